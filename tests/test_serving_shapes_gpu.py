"""The serving operators at the launch shapes that large batches take, against the same plain 64-bit forms
and bounds as test_serving_gpu.py: prompts cut into pieces, steps whose threads take four entries."""
import pytest
import torch

import serving_ref as R
from test_serving_gpu import DT, SENTINEL, Maker, cu_of, i32, scan_inputs, scan_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_61_amd as ssm
    ssm.load_library()


@pytest.fixture(scope="module")
def ssm():
    import selective_state_space_61_amd as m
    return m


@pytest.mark.parametrize("n", [1, 8, 16, 64])
@pytest.mark.parametrize("hint", [0, 5])
def test_scan_packed_infinite_state_stays(ssm, n, hint):
    """A state that became infinite stays so, in pieces (hint 0) as in one: no step's decay is zero here, but that
    of a whole piece is."""
    dim, rows, at = 40, 700, 300
    assert (ssm.ssm_scan_packed_workspace(rows, 1, hint, dim, n, torch.float32) > 0) == (hint == 0)
    m = Maker(n)
    d = scan_inputs(m, rows, dim, n, torch.float32, 0, False, False, False)
    d["A"] = -(1 + 15 * torch.arange(n, device="cuda") / max(n - 1, 1)).repeat(dim, 1).contiguous()
    if n == 1:
        d["A"] -= 11.0  # a piece's decay is zero for its one state too
    d["B"], d["C"] = d["B"].abs() + 0.1, d["C"].abs() + 0.1
    d["x"][at, 3:21] = float("inf")
    pool = torch.zeros(1, dim, n, device="cuda")
    y = ssm.ssm_scan_packed_fwd(d["x"], d["delta"], d["A"], d["B"], d["C"], cu_of([rows]), delta_softplus=True, cache=pool,
                                max_seqlen=hint)
    assert (y[at:, 3:21] == float("inf")).all() and (pool[0, 3:21] == float("inf")).all()
    d["x"][at, 3:21] = 0.0
    ref, err, h, eh = scan_ref(d, 0, rows, True, torch.zeros(dim, n, dtype=torch.float64))
    R.check(y[:at], ref[:at], err[:at], torch.float32, "before")
    others = [c for c in range(dim) if not 3 <= c < 21]
    R.check(y[:, others], ref[:, others], err[:, others], torch.float32, "the other channels")
    R.check(pool[0, others], h[others], eh[others], torch.float32, "their states")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cached", [True, False])
@pytest.mark.parametrize("batch,dim", [(5, 70), (250, 5120)])
def test_conv_step_of_width_one_skips_padding(ssm, batch, dim, cached, dtype):
    """Without windows too an entry without a slot keeps its row of y; without a cache every slot that is not
    negative counts."""
    m, dt, nslots = Maker(dim), DT[dtype], batch + 1
    x, w, b = m.normal((batch, dim), dt), m.normal((dim, 1)), m.normal((dim,))
    slots = list(range(batch))
    slots[1], slots[2], slots[batch - 1] = -1, nslots, 2_000_000_000
    pool = torch.empty(nslots, dim, 0, dtype=dt, device="cuda") if cached else None
    y = torch.full((batch, dim), SENTINEL, dtype=dt, device="cuda")
    ssm.ssm_causal_conv1d_update_cache(pool, i32(slots), x, w, b, y=y)
    ref, err = R.conv_rows(R.f64(x), R.f64(w), R.f64(b), True)
    live = [i for i, s in enumerate(slots) if 0 <= s and (s < nslots or not cached)]
    R.check(y[live], ref[live], err[live], dt, f"{len(live)} entries")
    assert (y[[i for i in range(batch) if i not in live]] == SENTINEL).all()
