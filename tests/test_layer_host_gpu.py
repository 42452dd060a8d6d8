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
