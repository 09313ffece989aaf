"""The serving operators at the launch shapes that large batches take, against the same plain 64-bit forms
and bounds as test_serving_gpu.py: the convolution's tiles of 32 rows, steps whose threads take four entries,
prompts cut into pieces at every dstate."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_serving_gpu import DT, SENTINEL, Maker, conv_case, cu_of, i32, scan_case, scan_inputs, scan_ref

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


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ---- the convolution's tiles of 32 rows ---------------------------------------------------------------

# starts one to three rows before a tile's end (31, 62, 93), sequences shorter than the window before and at a
# border, none, one of many tiles, a ragged last tile
TILES = [31, 31, 31, 1, 1, 1, 2, 30, 0, 29, 3, 200, 1100, 0, 227]


@pytest.mark.parametrize("width", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype,dim,gap", [("bf16", 5113, 0), ("bf16", 5120, 16), ("f32", 2570, 0)])
def test_conv_packed_large_tiles(ssm, dtype, dim, gap, width):
    total = sum(TILES)
    tiles = -(-total // 32)
    blocks = -(-(-(-dim // (2 if dtype == "bf16" else 1))) // 256)
    assert tiles * blocks >= 2 * cus() and len(TILES) <= tiles and total % 32  # what makes the tiles large
    conv_case(ssm, TILES, dim, width, dtype, gap=gap)


def test_conv_packed_large_tiles_behind_rows_of_no_sequence(ssm):
    conv_case(ssm, TILES, 5120, 4, "bf16", first=33, tail=70, slots=[-1, 3, 16, 0, 2_000_000_000] + list(range(4, 14)))


# ---- steps whose threads take four entries --------------------------------------------------------------


def padded_slots(batch, nslots):
    """Each entry its own slot, entries without one inside, at the start and at the end of groups of four."""
    s = [int(v) for v in np.random.default_rng(batch).permutation(nslots)[:batch]]
    for i, bad in zip((0, 5, 6, 11, batch - 1), (-1, nslots, -7, 2_000_000_000, -1)):
        s[i] = bad
    return s


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("batch,dim,gap", [(250, 5120, 8), (251, 5113, 0)])
def test_conv_step_four_entries_a_thread(ssm, batch, dim, gap, width, dtype):
    assert -(-dim // 1024) * -(-batch // 4) >= cus()
    m, dt, nslots = Maker(dim + width), DT[dtype], batch + 9
    slots = padded_slots(batch, nslots)
    x, w, b = m.rows(batch, dim, dt, gap), m.normal((dim, width)), m.normal((dim,))
    pool = m.normal((nslots, dim, width - 1), dt)
    before = pool.cpu().clone()
    y = torch.full((batch, dim + gap), SENTINEL, dtype=dt, device="cuda")[:, gap // 2:gap // 2 + dim]
    ssm.ssm_causal_conv1d_update_cache(pool, i32(slots), x, w, b, y=y)
    torch.cuda.synchronize()
    live = [i for i, s in enumerate(slots) if 0 <= s < nslots]
    at = [slots[i] for i in live]
    line = torch.cat([before[at].double().transpose(1, 2), R.f64(x)[live][:, None]], 1)  # (entries, width, dim)
    ref, err = R.conv_rows(line.transpose(0, 1).reshape(width, -1), R.f64(w).repeat(len(live), 1),
                           R.f64(b).repeat(len(live)), True)
    R.check(y[live].reshape(1, -1), ref, err, dt, f"{len(live)} entries")
    assert (y[[i for i in range(batch) if i not in live]] == SENTINEL).all()
    before[at] = line[:, 1:].transpose(1, 2).to(dt)
    assert torch.equal(pool.cpu(), before)


@pytest.mark.parametrize("n,dtype,cdtype", [(n, *t) for n in (1, 2, 4, 8, 16, 32, 64) for t in (("bf16", "f32"), ("f32", "bf16"))]
                         + [(16, "f32", "f32"), (16, "bf16", "bf16")])
@pytest.mark.parametrize("dim,gap", [(5120, 16), (5113, 0)])
def test_scan_step_four_entries_a_thread(ssm, dim, gap, n, dtype, cdtype):
    dt, cdt = DT[dtype], DT[cdtype]
    lanes = n // (min(n, 8) if cdtype == "bf16" else min(n, 4))
    blocks = -(-dim * lanes // 256)
    batch = max(4 * -(-cus() // blocks), 12) + 2
    assert blocks * -(-batch // 4) >= cus() and batch % 4
    m, nslots = Maker(dim + n), batch + 5
    slots = padded_slots(batch, nslots)
    d = scan_inputs(m, batch, dim, n, dt, gap, True, True, True)
    pool = m.normal((nslots, dim, n), cdt)
    before = pool.clone()
    y = torch.full((batch, dim + gap), SENTINEL, dtype=dt, device="cuda")[:, gap // 2:gap // 2 + dim]
    ssm.ssm_state_update_cache(pool, i32(slots), d["x"], d["delta"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"],
                               delta_bias=d["delta_bias"], delta_softplus=True, y=y)
    torch.cuda.synchronize()
    kept = torch.ones(nslots, dtype=torch.bool)
    for i, s in enumerate(slots):
        if not 0 <= s < nslots:
            assert (y[i] == SENTINEL).all()
            continue
        ref, err, h, eh = scan_ref(d, i, i + 1, True, R.f64(before[s]))
        R.check(y[i:i + 1], ref, err, dt, f"entry {i}")
        R.check(pool[s], h, eh, cdt, f"state {i}")
        kept[s] = False
    assert torch.equal(pool[kept.cuda()], before[kept.cuda()])


# ---- prompts cut into pieces ------------------------------------------------------------------------------


def assert_cut(ssm, lens, extra, hint, dim, n, dtype):
    """The launch has pieces: they are what the workspace is for."""
    assert ssm.ssm_scan_packed_workspace(sum(lens) + extra, len(lens), hint, dim, n, DT[dtype]) > 0


@pytest.mark.parametrize("n", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("lens,hint", [([1500], 0), ([700, 3, 801], 801), ([300, 0, 17, 400], 400)], ids=str)
@pytest.mark.parametrize("dtype,cdtype", [("f32", "bf16"), ("bf16", "f32")])
def test_scan_packed_pieces(ssm, lens, hint, n, dtype, cdtype):
    # the first sequence, and every third after it, goes on from its slot
    for dim, gap, first, tail in ((72, 0, 2, 3), (33, 5, 0, 0), (3, 0, 1, 0)):
        assert_cut(ssm, lens, first + tail, hint, dim, n, dtype)
        scan_case(ssm, lens, dim, n, dtype, cdtype, max_seqlen=hint, gap=gap, first=first, tail=tail)


@pytest.mark.parametrize("n", [1, 16, 64])
def test_scan_packed_pieces_variants(ssm, n):
    lens = [700, 3, 801]
    for kw in (dict(cache=False), dict(initial=False), dict(z=False, D=False), dict(slots=[1, -1, 2_000_000_000])):
        assert_cut(ssm, lens, 0, 0, 40, n, "bf16")
        scan_case(ssm, lens, 40, n, "bf16", **kw)


@pytest.mark.parametrize("n", [2, 16, 32])
def test_scan_packed_pieces_whatever_the_workspace_holds(ssm, n):
    m, lens, dim = Maker(n), [500, 1, 620], 40
    d = scan_inputs(m, sum(lens), dim, n, torch.bfloat16, 0, True, True, True)
    size = ssm.ssm_scan_packed_workspace(sum(lens), len(lens), 620, dim, n, torch.bfloat16)
    assert size > 0
    pool = m.normal((3, dim, n))
    got = []
    for fill in (0, 255):  # 255: every float a NaN
        cache = pool.clone()
        y = ssm.ssm_scan_packed_fwd(d["x"], d["delta"], d["A"], d["B"], d["C"], cu_of(lens), D=d["D"], z=d["z"],
                                    delta_bias=d["delta_bias"], delta_softplus=True, cache=cache, max_seqlen=620,
                                    has_initial=torch.ones(3, dtype=torch.bool, device="cuda"),
                                    workspace=torch.full((size,), fill, dtype=torch.uint8, device="cuda"))
        got.append((y, cache))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.isfinite(got[0][0]).all() and torch.isfinite(got[0][1]).all()


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
