"""Decode steps whose context is no longer than the rectification band: the
cached summaries AS_{1:p-r} are empty, so a hit attends its band and tail
alone, and the summaries it appends are empty or start from nothing.  Every
output and every ring entry is finite, and the trajectories match the
oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from harness import TOL, Problem, compare, gpu_trajectory, oracle_trajectory  # noqa: E402
from long_context_decode_gb300 import mac  # noqa: E402
from long_context_decode_gb300.workloads import BF16, F32, Workload  # noqa: E402
from oracle import mac_oracle as O  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_decode_gb300 import build as b
    b.build()
    mac.load()


# tau: hits wherever there is a candidate, or misses among them, so that a summary started by a miss is met by hits
@pytest.mark.parametrize("tau", [-1.0, 0.05])
@pytest.mark.parametrize("Hq,Hkv,dtype,paged,aux,seed_rows", [
    (8, 2, BF16, True, False, 0), (8, 2, BF16, False, True, 0), (4, 4, F32, True, False, 0), (4, 2, BF16, False, False, 5),
    (4, 1, F32, False, True, 5), (16, 2, BF16, True, False, 0), (8, 1, F32, False, False, 5)])
def test_hits_within_the_band(Hq, Hkv, dtype, paged, aux, seed_rows, tau):
    # from no context, one inside the band and one that leaves it on the way
    w = Workload("short", 3, Hq, Hkv, 128, [seed_rows, 11, 29], 16, 32, tau, dtype, 0, 24, 31, "ar1_jump", "normal")
    P = Problem(w, n_seed=seed_rows, paged=paged)
    gpu, st, layer = gpu_trajectory(P, w.n_steps, aux=aux)
    assert all(np.isfinite(out).all() for out, _ in gpu)
    assert torch.isfinite(layer.ring_view("o")).all() and not torch.isnan(layer.ring_view("lse")).any()
    ref = oracle_trajectory(P, w.n_steps)
    c = compare(gpu, ref, O.threshold_sq(128, w.tau))
    assert st == 0 and c["mismatched"] == 0 and c["max_err"] <= TOL, c
    assert c["hits"] > 0
    layer.release()
