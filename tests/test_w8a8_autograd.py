"""The 8-bit calls beside autograd: they are forward only, say so where a gradient would be lost, and
mark the caller's tensors that they write as changed."""
import pytest

torch = pytest.importorskip("torch")
rl = pytest.importorskip("rotated_linear_amd", reason="libparo.so not built")


def calls(device):
    """(name, call, tensors by name, the names whose gradient would be lost) with a call of those tensors."""
    M, D, N = 3, 256, 10
    torch.manual_seed(3)

    def t(*shape, dtype=torch.float16):
        return torch.ones(shape, dtype=dtype, device=device)

    def q(*shape):
        return torch.ones(shape, dtype=torch.int8, device=device)

    norm = {"x": t(M, D), "gamma": t(D), "residual": t(M, D), "residual_out": t(M, D)}
    out8 = {"q": q(M, D), "scales": t(M, dtype=torch.float32)}
    yield ("rmsnorm_q8", lambda x, gamma, residual, residual_out, q, scales:
           rl.paro_rmsnorm_q8(x, gamma, 1e-6, residual=residual, out=(q, scales), residual_out=residual_out), {**norm, **out8})
    yield ("rmsnorm", lambda x, gamma, residual, residual_out, out:
           rl.paro_rmsnorm(x, gamma, 1e-6, residual=residual, out=out, residual_out=residual_out), {**norm, "out": t(M, D)})
    yield ("quantize", lambda x, q, scales: rl.paro_quantize_q8(x, out=(q, scales)), {"x": t(M, D), **out8})
    yield ("pack", lambda W, qweight, scales: rl.paro_pack_weights_q8(W, out=(qweight, scales)),
           {"W": t(N, D), "qweight": q(N, D), "scales": t(N, dtype=torch.float32)})
    yield ("dequantize", lambda q, scales, out: rl.paro_dequantize_q8(q, scales, out=out),
           {"q": q(M, D), "scales": t(M, dtype=torch.float32), "out": t(M, D)})
    for gated in (False, True):
        f = rl.paro_w8a8_gated_linear if gated else rl.paro_w8a8_linear
        yield ("gated" if gated else "linear", lambda x, x_scales, qweight, w_scales, out, f=f: f(x, x_scales, qweight, w_scales, out=out),
               {"x": q(M, D), "x_scales": t(M, dtype=torch.float32), "qweight": q(N, D), "w_scales": t(N, dtype=torch.float32),
                "out": t(M, N // 2 if gated else N)})


WRITTEN_BY = {"rmsnorm_q8": {"residual_out", "q", "scales"}, "rmsnorm": {"residual_out", "out"}, "quantize": {"q", "scales"},
              "pack": {"qweight", "scales"}, "dequantize": {"out"}, "linear": {"out"}, "gated": {"out"}}


def refuses(device):
    for name, call, given in calls(device):
        for which, t in given.items():
            if not t.is_floating_point() or which == "W":
                continue
            asked = {k: v.clone().requires_grad_(k == which) for k, v in given.items()}
            with pytest.raises(RuntimeError, match=f"{which} requires a gradient and this call is forward only"):
                call(**asked)
            yield name, call, asked


def test_a_gradient_that_would_be_lost_is_refused():
    """Before the device is looked at: CPU tensors show it. Under no_grad the next check speaks."""
    n = 0
    for name, call, asked in refuses("cpu"):
        with torch.no_grad(), pytest.raises(ValueError, match="must live on the GPU"):
            call(**asked)
        n += 1
    assert n == 5 + 5 + 2 + 1 + 2 + 3 + 3
    with pytest.raises(ValueError, match="must live on the GPU"):  # packing a parameter is nothing to refuse
        rl.paro_pack_weights_q8(torch.nn.Parameter(torch.ones(4, 256, dtype=torch.float16)))


@pytest.mark.gpu
def test_a_gradient_that_would_be_lost_is_refused_on_the_gpu():
    for name, call, asked in refuses("cuda"):
        with torch.no_grad():
            call(**asked)
    q, s = rl.paro_pack_weights_q8(torch.nn.Parameter(torch.ones(4, 256, dtype=torch.float16, device="cuda")))
    assert not q.requires_grad and not s.requires_grad and int(q.sum()) == 127 * 4 * 256
    torch.cuda.synchronize()


class Unusual(torch.Tensor):
    pass


@pytest.mark.gpu
@pytest.mark.parametrize("way", ["compiled", "checked"])
def test_written_tensors_count_as_changed(way):
    """Through the compiled binding and through the checked way (a tensor subclass takes it)."""
    for name, call, given in calls("cuda"):
        if way == "checked":
            first = next(iter(given))
            given[first] = given[first].as_subclass(Unusual)
        before = {k: v._version for k, v in given.items()}
        call(**given)
        after = {k: v._version for k, v in given.items()}
        assert {k for k in given if after[k] != before[k]} == WRITTEN_BY[name], name
    # what autograd keeps of a stream that a call then updates in place
    w = torch.ones(2, 256, dtype=torch.float16, device="cuda", requires_grad=True)
    stream = torch.ones(2, 256, dtype=torch.float16, device="cuda")
    kept = (w * stream).sum()
    x = stream.clone().as_subclass(Unusual) if way == "checked" else stream.clone()
    rl.paro_rmsnorm_q8(x, torch.ones(256, dtype=torch.float16, device="cuda"), residual=stream, residual_out=stream)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.backward()
    with torch.inference_mode():  # tensors without a version counter
        given = {k: v.clone() for k, v in next(calls("cuda"))[2].items()}
    next(calls("cuda"))[1](**given)
    torch.cuda.synchronize()
