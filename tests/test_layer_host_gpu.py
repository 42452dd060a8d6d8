"""Calls of the layer operators from several host threads, after a failed call, and without memory for scratch."""
import ctypes
import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_gb300 as g
    g.lib()
    yield g
    assert g.device_status(0) == 0


# two lengths of row that take one instantiation of a kernel with different amounts of shared memory
@pytest.mark.parametrize("D", [(32768, 16392), (16001, 12299)])
def test_rows_of_different_lengths_from_two_threads(gdn, D):
    """No thread's call depends on the shared memory that another's needs."""
    errors = []
    x = [torch.ones(1, d, dtype=torch.bfloat16, device="cuda") for d in D]
    w = [torch.ones(d, device="cuda") for d in D]
    out = [torch.empty_like(t) for t in x]
    streams = [torch.cuda.Stream() for _ in D]
    torch.cuda.synchronize()
    start = threading.Barrier(len(D))

    def work(i):
        start.wait()
        try:
            for _ in range(20000):
                gdn.rmsnorm_residual(x[i], w[i], out=out[i], stream=streams[i])
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(D))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for o in out:
        assert (o == 1).all()


def _fail_once(call):
    """Runs ``call(stream)`` on a stream whose capture has been invalidated by a forbidden call: its launch is refused."""
    rt = ctypes.CDLL("libcudart.so.%s" % torch.version.cuda.split(".")[0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(ctypes.c_void_p(s.cuda_stream), 0) == 0
    assert rt.cudaDeviceSynchronize() != 0
    try:
        call(s)
    finally:
        graph = ctypes.c_void_p()
        assert rt.cudaStreamEndCapture(ctypes.c_void_p(s.cuda_stream), ctypes.byref(graph)) != 0
        rt.cudaGetLastError()


@pytest.mark.parametrize("failing", ["linear", "linear_parts", "norm"])
def test_a_failed_call_does_not_fail_the_next(gdn, failing):
    """A refused launch is that call's error only: the products that lay their operands out anew, the older entry points
    and the norm work afterwards."""
    gen = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    xf, wf = rand(300, 1024), rand(1024, 1024)
    xb, wb = rand(700, 1001).bfloat16(), rand(1001, 1001).bfloat16()
    cx, cw = rand(1, 256, 16).bfloat16(), rand(256, 4)
    n, nw = rand(4, 256), torch.ones(256, device="cuda")
    out, outn = torch.empty(300, 1024, device="cuda"), torch.empty_like(n)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    calls = [lambda: gdn.linear(xf, wf), lambda: gdn.linear(xb, wb), lambda: gdn.conv1d_prefill(cx, cw)[0],
             lambda: gdn.rmsnorm_residual(n, nw)[0]]
    ref = [c() for c in calls]

    def fail(s):
        with pytest.raises(gdn.GdnError) as e:
            if failing == "norm":
                gdn.rmsnorm_residual(n, nw, out=outn, stream=s)
            elif failing == "linear":
                gdn.linear(xf, wf, out=out, force_ffma=True, stream=s)
            else:
                d = gdn.GdnLinearDims(300, 1024, 1024, gdn.GDN_F32, gdn.GDN_F32, 0, 0)
                gdn._binding._check(gdn.lib().gdn_linear_ws(xf.data_ptr(), None, wf.data_ptr(), None, None, None, out.data_ptr(),
                                                           ctypes.byref(d), ws.data_ptr(), ws.numel(), s.cuda_stream))
        assert e.value.code == gdn.GDN_ERR_CUDA
    for c, r in zip(calls, ref):
        _fail_once(fail)
        assert torch.equal(c(), r)


def test_products_without_memory_for_scratch(gdn, monkeypatch):
    """Operands that are laid out anew where torch has no memory for it: the call still gives its result."""
    gen = torch.Generator("cuda").manual_seed(1)
    x, w = (torch.randn(n, 2048, generator=gen, device="cuda") for n in (4096, 2048))
    xb, wb = x.view(-1)[:4001 * 2047].view(4001, 2047).bfloat16(), w.view(-1)[:2047 * 2048].view(2047, 2048).bfloat16()
    calls = (lambda: gdn.linear(x, w, weight_layout="nk"), lambda: gdn.linear(xb, wb))
    ref = [c() for c in calls]
    empty, refused = gdn._binding._layer_empty, []

    def short_of_memory(shape, dtype, device, stream):
        if dtype is torch.uint8:
            refused.append(shape)
            raise torch.OutOfMemoryError("no memory for scratch")
        return empty(shape, dtype, device, stream)
    monkeypatch.setattr(gdn._binding, "_layer_empty", short_of_memory)
    for c, r in zip(calls, ref):
        assert torch.equal(c(), r)
    assert len(refused) == 2
