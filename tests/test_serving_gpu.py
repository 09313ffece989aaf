"""The serving operators on the GPU, through the binding and the C ABI, against their plain 64-bit
forms (serving_ref.py, whose bounds count the roundings): packed prompts, steps on a cache of slots,
states set aside in 8 bits, and a run of them together."""
import numpy as np
import pytest
import torch

import serving_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SENTINEL = -77.0


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


class Maker:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def normal(self, shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=self.g) * scale).to(dtype).cuda()

    def rows(self, n, width, dtype, gap=0, scale=1.0):
        """(n, width), its rows `gap` elements apart from one another (and off a 16-byte boundary)."""
        if not gap:
            return self.normal((n, width), dtype, scale)
        return self.normal((n, width + gap), dtype, scale)[:, gap // 2:gap // 2 + width]

    def A(self, dim, n):
        return (-torch.rand(dim, n, generator=self.g) * 15 - 0.05).cuda()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cu_of(lens, first=0):
    return i32([first] + [first + int(c) for c in np.cumsum(lens)])


# ---- the convolution ------------------------------------------------------------------------------

# lengths; the tiles are 32 rows, so starts one to three rows before a tile's end are here too
PROMPTS = [[1], [5], [31, 40], [30, 3, 40], [29, 2, 1, 1, 70], [32, 32], [0, 3, 0, 70, 1, 0], [33, 1, 1, 1, 2, 100], [97]]


def conv_case(ssm, lens, dim, width, dtype, *, gap=0, first=0, tail=0, initial=True, cache=True, bias=True, act=True,
              slots=None, seed=0):
    m = Maker(seed + 13 * dim + width)
    dt = DT[dtype]
    total, n = first + sum(lens) + tail, len(lens)
    x = m.rows(total, dim, dt, gap)
    y = torch.full((total, dim + gap), SENTINEL, dtype=dt, device="cuda")[:, gap // 2:gap // 2 + dim]
    w, b = m.normal((dim, width)), m.normal((dim,)) if bias else None
    nslots = n + 2
    slots = list(np.random.default_rng(seed).permutation(nslots)[:n]) if slots is None else slots
    pool = m.normal((nslots, dim, width - 1), dt) if cache else None
    before = None if pool is None else pool.clone()
    init = [(i % 3) != 1 for i in range(n)] if initial and cache else None
    got = ssm.ssm_causal_conv1d_packed_fwd(
        x, w, cu_of(lens, first), b, act, cache=pool, cache_slots=i32(slots) if cache else None,
        has_initial=None if init is None else torch.tensor(init, device="cuda"), y=y)
    torch.cuda.synchronize()
    assert got is y
    expect = None if pool is None else before.cpu().clone()
    r0 = first
    for i, L in enumerate(lens):
        ok = cache and 0 <= slots[i] < nslots
        win = torch.zeros(width - 1, dim, dtype=torch.float64)
        if ok and init is not None and init[i]:
            win = R.f64(before[slots[i]]).T
        line = torch.cat([win, R.f64(x[r0:r0 + L])])
        ref, err = R.conv_rows(line, R.f64(w), R.f64(b), act)
        if L:
            R.check(y[r0:r0 + L], ref, err, dt, f"seq {i} of {L} rows")
            if ok:
                expect[slots[i]] = line[line.shape[0] - (width - 1):].T.to(dt)
        r0 += L
    assert (y[:first] == SENTINEL).all() and (y[r0:] == SENTINEL).all(), "rows of no sequence were written"
    if cache:
        assert torch.equal(pool.cpu(), expect), "windows differ"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", PROMPTS, ids=str)
def test_conv_packed_lengths(ssm, lens, dtype):
    conv_case(ssm, lens, 70, 4, dtype, first=3, tail=5)


@pytest.mark.parametrize("width", [1, 2, 3, 4])
@pytest.mark.parametrize("dim,gap", [(1, 0), (8, 6), (513, 0), (600, 9), (1030, 2)])
def test_conv_packed_widths_and_strides(ssm, dim, gap, width):
    conv_case(ssm, [30, 3, 40], dim, width, "bf16" if dim % 2 else "f32", gap=gap)
    conv_case(ssm, [1, 66], dim, width, "bf16", gap=gap)


@pytest.mark.parametrize("variant", ["no_initial", "no_cache", "no_bias", "no_silu", "no_slot", "past_slots"])
def test_conv_packed_variants(ssm, variant):
    lens = [31, 5, 40]
    slots = {"no_slot": [2, -1, 0], "past_slots": [1, 2_000_000_000, 5]}.get(variant)
    conv_case(ssm, lens, 64, 4, "bf16", initial=variant != "no_initial", cache=variant != "no_cache",
              bias=variant != "no_bias", act=variant != "no_silu", slots=slots, tail=1)


def test_conv_packed_many_sequences(ssm):
    # more sequences than a wave has lanes, and lengths of one
    conv_case(ssm, [1] * 150 + [0] * 70 + [2, 35], 24, 4, "bf16", first=1, tail=2)


# ---- the scan ---------------------------------------------------------------------------------------


def scan_inputs(m, total, dim, n, dt, gap, z, D, bias):
    return dict(x=m.rows(total, dim, dt, gap), delta=m.rows(total, dim, dt, gap, 0.5), A=m.A(dim, n),
                B=m.rows(total, n, dt, gap), C=m.rows(total, n, dt, gap), D=m.normal((dim,)) if D else None,
                z=m.rows(total, dim, dt, gap) if z else None, delta_bias=m.normal((dim,), scale=2.0) - 2 if bias else None)


def scan_ref(d, lo, hi, softplus, h0):
    pick = lambda k: None if d[k] is None else R.f64(d[k][lo:hi])  # noqa: E731
    return R.scan_steps(pick("x"), pick("delta"), R.f64(d["A"]), pick("B"), pick("C"), R.f64(d["D"]), pick("z"),
                        R.f64(d["delta_bias"]), softplus, h0)


def scan_case(ssm, lens, dim, n, dtype, cdtype="f32", *, gap=0, first=0, tail=0, initial=True, cache=True, z=True,
              D=True, bias=True, softplus=True, slots=None, max_seqlen=0, seed=0, edit=None):
    m = Maker(seed + 17 * dim + n)
    dt, cdt = DT[dtype], DT[cdtype]
    total, ns = first + sum(lens) + tail, len(lens)
    d = scan_inputs(m, total, dim, n, dt, gap, z, D, bias)
    if not softplus:
        d["delta"] = d["delta"].abs() * 0.2
    y = torch.full((total, dim + gap), SENTINEL, dtype=dt, device="cuda")[:, gap // 2:gap // 2 + dim]
    nslots = ns + 2
    slots = [int(s) for s in np.random.default_rng(seed).permutation(nslots)[:ns]] if slots is None else slots
    pool = m.normal((nslots, dim, n), cdt) if cache else None
    before = None if pool is None else pool.clone()
    init = [(i % 3) != 1 for i in range(ns)] if initial and cache else None
    if edit:
        edit(d)
    got = ssm.ssm_scan_packed_fwd(
        d["x"], d["delta"], d["A"], d["B"], d["C"], cu_of(lens, first), D=d["D"], z=d["z"], delta_bias=d["delta_bias"],
        delta_softplus=softplus, cache=pool, cache_slots=i32(slots) if cache else None,
        has_initial=None if init is None else torch.tensor(init, device="cuda"), max_seqlen=max_seqlen, y=y)
    torch.cuda.synchronize()
    assert got is y
    touched = set()
    r0 = first
    for i, L in enumerate(lens):
        ok = cache and 0 <= slots[i] < nslots
        h0 = torch.zeros(dim, n, dtype=torch.float64)
        if ok and init is not None and init[i]:
            h0 = R.f64(before[slots[i]])
        if L:
            ref, err, h, eh = scan_ref(d, r0, r0 + L, softplus, h0)
            R.check(y[r0:r0 + L], ref, err, dt, f"seq {i} of {L} rows")
            if ok:
                R.check(pool[slots[i]], h, eh, cdt, f"state {i}")
                touched.add(int(slots[i]))
        r0 += L
    assert (y[:first] == SENTINEL).all() and (y[r0:] == SENTINEL).all(), "rows of no sequence were written"
    for s in range(nslots if cache else 0):
        if s not in touched:
            assert torch.equal(pool[s], before[s]), f"slot {s} was written"


@pytest.mark.parametrize("dtype,cdtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("lens", PROMPTS, ids=str)
def test_scan_packed_lengths(ssm, lens, dtype, cdtype):
    scan_case(ssm, lens, 56, 16, dtype, cdtype, first=3, tail=5)


@pytest.mark.parametrize("n", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("dim,gap", [(1, 0), (40, 6), (97, 5), (130, 16)])
def test_scan_packed_states_and_strides(ssm, n, dim, gap):
    scan_case(ssm, [18, 1, 35], dim, n, "bf16", "f32", gap=gap)
    scan_case(ssm, [18, 1, 35], dim, n, "f32", "bf16", gap=gap)


@pytest.mark.parametrize("variant", ["no_initial", "no_cache", "no_bias", "no_softplus", "no_z", "no_D", "no_slot",
                                     "past_slots", "plain_steps"])
def test_scan_packed_variants(ssm, variant):
    slots = {"no_slot": [2, -1, 0], "past_slots": [1, 2_000_000_000, 5]}.get(variant)
    for n in (16, 8):
        scan_case(ssm, [31, 5, 40], 64, n, "bf16", initial=variant != "no_initial", cache=variant != "no_cache",
                  bias=variant not in ("no_bias", "plain_steps"), softplus=variant not in ("no_softplus", "plain_steps"), z=variant != "no_z",
                  D=variant != "no_D", slots=slots, tail=1)


def test_scan_packed_many_sequences(ssm):
    scan_case(ssm, [1] * 150 + [0] * 70 + [2, 35], 24, 16, "bf16", first=1, tail=2)


# long enough to be cut into pieces where the rule says so; a wrong hint changes only the launch
@pytest.mark.parametrize("dtype,cdtype", [("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("lens,hint", [([1500], 0), ([700, 3, 801], 801), ([1100], 5), ([40, 900], 2_000_000)], ids=str)
def test_scan_packed_long(ssm, lens, hint, dtype, cdtype):
    scan_case(ssm, lens, 72, 16, dtype, cdtype, max_seqlen=hint, first=2, tail=3)
    scan_case(ssm, lens, 33, 8, dtype, cdtype, max_seqlen=hint, gap=3)


@pytest.mark.parametrize("lens", [[20, 20, 20], [700, 33, 700]], ids=str)
def test_scan_packed_nan_stays_in_its_sequence(ssm, lens):
    # every input of the middle sequence, and the rows of no sequence, are NaN or infinite
    def edit(d):
        for k in ("x", "delta", "B", "C", "z"):
            d[k][1 + lens[0]:1 + lens[0] + lens[1]] = float("nan")
            d[k][0] = float("inf")
            d[k][-1] = float("nan")
    m = Maker(1)
    d = scan_inputs(m, sum(lens) + 2, 48, 16, torch.bfloat16, 0, True, True, True)
    edit(d)
    pool = torch.zeros(3, 48, 16, device="cuda")
    y = ssm.ssm_scan_packed_fwd(d["x"], d["delta"], d["A"], d["B"], d["C"], cu_of(lens, 1), D=d["D"], z=d["z"],
                                delta_bias=d["delta_bias"], delta_softplus=True, cache=pool, max_seqlen=max(lens))
    r = 1
    for i, L in enumerate(lens):
        if i == 1:
            assert torch.isnan(y[r:r + L]).all() and torch.isnan(pool[1]).all()
        else:
            ref, err, h, eh = scan_ref(d, r, r + L, True, torch.zeros(48, 16, dtype=torch.float64))
            R.check(y[r:r + L], ref, err, torch.bfloat16, f"seq {i}")
            R.check(pool[i], h, eh, torch.float32, f"state {i}")
        r += L


def test_scan_packed_matches_the_dense_scan(ssm):
    # equal lengths packed one behind another are the dense scan's batch
    m = Maker(5)
    d = scan_inputs(m, 4 * 200, 160, 16, torch.bfloat16, 0, True, True, True)
    pool = torch.full((4, 160, 16), SENTINEL, device="cuda")
    y = ssm.ssm_scan_packed_fwd(d["x"], d["delta"], d["A"], d["B"], d["C"], cu_of([200] * 4), D=d["D"], z=d["z"],
                                delta_bias=d["delta_bias"], delta_softplus=True, cache=pool)
    sh = lambda t: t.view(4, 200, -1)  # noqa: E731
    y2, st = ssm.ssm_scan_fwd(sh(d["x"]), sh(d["delta"]), d["A"], sh(d["B"]), sh(d["C"]), D=d["D"], z=sh(d["z"]),
                              delta_bias=d["delta_bias"], delta_softplus=True)
    # both are within their bound of the same values
    for b in range(4):
        ref, err, h, eh = scan_ref(d, 200 * b, 200 * b + 200, True, torch.zeros(160, 16, dtype=torch.float64))
        R.check(y[200 * b:200 * b + 200], ref, err, torch.bfloat16, f"packed {b}")
        R.check(y2[b], ref, err, torch.bfloat16, f"dense {b}")
        R.check(pool[b], h, eh, torch.float32, f"packed state {b}")


# ---- single tokens ----------------------------------------------------------------------------------


def slots_of(batch, nslots, pad, seed=0):
    s = [int(v) for v in np.random.default_rng(seed).permutation(nslots)[:batch]]
    for i in pad:
        s[i] = (-1, nslots, 2_000_000_000)[i % 3]
    return s


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [1, 2, 3, 4])
@pytest.mark.parametrize("batch,dim,gap", [(1, 1, 0), (3, 64, 0), (9, 70, 4), (5, 1029, 3), (17, 2048, 8)])
def test_conv_step_cache(ssm, batch, dim, gap, width, dtype):
    m = Maker(dim + width)
    dt = DT[dtype]
    nslots = batch + 3
    pad = [batch // 2] if batch > 2 and width > 1 else []
    slots = slots_of(batch, nslots, pad)
    x, w, b = m.rows(batch, dim, dt, gap), m.normal((dim, width)), m.normal((dim,))
    pool = m.normal((nslots, dim, width - 1), dt)
    before = pool.clone()
    y = torch.full((batch, dim + gap), SENTINEL, dtype=dt, device="cuda")[:, gap // 2:gap // 2 + dim]
    ssm.ssm_causal_conv1d_update_cache(pool, i32(slots), x, w, b, y=y)
    torch.cuda.synchronize()
    expect = before.cpu().clone()
    for i, s in enumerate(slots):
        if i in pad:
            assert (y[i] == SENTINEL).all()
            continue
        line = torch.cat([R.f64(before[s]).T, R.f64(x[i:i + 1])])
        ref, err = R.conv_rows(line, R.f64(w), R.f64(b), True)
        R.check(y[i:i + 1], ref, err, dt, f"entry {i}")
        expect[s] = line[1:].T.to(dt)
    assert torch.equal(pool.cpu(), expect)


@pytest.mark.parametrize("dtype,cdtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("n", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("batch,dim,gap", [(1, 1, 0), (3, 64, 0), (7, 70, 4), (21, 333, 3)])
def test_scan_step_cache(ssm, batch, dim, gap, n, dtype, cdtype):
    m = Maker(dim + n)
    dt, cdt = DT[dtype], DT[cdtype]
    nslots = batch + 3
    pad = [batch // 2] if batch > 2 else []
    slots = slots_of(batch, nslots, pad)
    d = scan_inputs(m, batch, dim, n, dt, gap, dim != 70, dim != 64, True)
    pool = m.normal((nslots, dim, n), cdt)
    before = pool.clone()
    y = torch.full((batch, dim + gap), SENTINEL, dtype=dt, device="cuda")[:, gap // 2:gap // 2 + dim]
    ssm.ssm_state_update_cache(pool, i32(slots), d["x"], d["delta"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"],
                               delta_bias=d["delta_bias"], delta_softplus=True, y=y)
    torch.cuda.synchronize()
    live = set()
    for i, s in enumerate(slots):
        if i in pad:
            assert (y[i] == SENTINEL).all()
            continue
        ref, err, h, eh = scan_ref(d, i, i + 1, True, R.f64(before[s]))
        R.check(y[i:i + 1], ref, err, dt, f"entry {i}")
        R.check(pool[s], h, eh, cdt, f"state {i}")
        live.add(s)
    for s in range(nslots):
        if s not in live:
            assert torch.equal(pool[s], before[s])


@pytest.mark.parametrize("dtype,cdtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("n", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("batch,heads,headdim,groups,gap", [(1, 1, 64, 1, 0), (4, 6, 20, 2, 0), (3, 4, 70, 4, 5),
                                                            (5, 3, 128, 1, 16)])
def test_ssd_step_cache(ssm, batch, heads, headdim, groups, gap, n, dtype, cdtype):
    m = Maker(heads * headdim + n)
    dt_, cdt = DT[dtype], DT[cdtype]
    nslots = batch + 2
    pad = [1] if batch > 2 else []
    slots = slots_of(batch, nslots, pad)
    x, z = (m.rows(batch, heads * headdim, dt_, gap).unflatten(1, (heads, headdim)) for _ in range(2))
    B, C = (m.rows(batch, groups * n, dt_, gap).unflatten(1, (groups, n)) for _ in range(2))
    dt = m.rows(batch, heads, dt_, gap, 0.5)
    A, D, bias = m.A(heads, 1)[:, 0].contiguous(), m.normal((heads,)), m.normal((heads,)) - 2
    if headdim == 20:
        z, D = None, None
    pool = m.normal((nslots, heads, headdim, n), cdt)
    before = pool.clone()
    y = torch.full((batch, heads * headdim + gap), SENTINEL, dtype=dt_, device="cuda")
    y = y[:, gap // 2:gap // 2 + heads * headdim].unflatten(1, (heads, headdim))
    ssm.ssm_ssd_state_update_cache(pool, i32(slots), x, dt, A, B, C, D=D, z=z, dt_bias=bias, dt_softplus=True, y=y)
    torch.cuda.synchronize()
    live = set()
    for i, s in enumerate(slots):
        if i in pad:
            assert (y[i] == SENTINEL).all()
            continue
        live.add(s)
        for h in range(heads):  # a head is a scan whose channels share dt, A, D
            g = h // (heads // groups)
            one = lambda t: R.f64(t[i, h])[None]  # noqa: E731
            dh = R.f64(dt[i, h]).expand(1, headdim)
            ref, err, st, es = R.scan_steps(one(x), dh, R.f64(A[h]).expand(headdim, n), R.f64(B[i, g])[None],
                                            R.f64(C[i, g])[None], None if D is None else R.f64(D[h]),
                                            None if z is None else one(z), R.f64(bias[h]).expand(headdim), True,
                                            R.f64(before[s, h]))
            R.check(y[i, h][None], ref, err, dt_, f"entry {i} head {h}")
            R.check(pool[s, h], st, es, cdt, f"state {i} head {h}")
    for s in range(nslots):
        if s not in live:
            assert torch.equal(pool[s], before[s])


def test_steps_without_slots_take_them_in_order(ssm):
    m = Maker(3)
    d = scan_inputs(m, 5, 32, 16, torch.bfloat16, 0, True, True, True)
    a = m.normal((7, 32, 16))
    b = a.clone()
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"], delta_softplus=True)
    args = (d["x"], d["delta"], d["A"], d["B"], d["C"])
    y1 = ssm.ssm_state_update_cache(a, None, *args, **kw)
    y2 = ssm.ssm_state_update_cache(b, i32(list(range(5))), *args, **kw)
    assert torch.equal(y1, y2) and torch.equal(a, b)


def test_step_batch_beyond_the_grid(ssm):
    # more entries than a launch has workgroups in a dimension
    m = Maker(8)
    n = 70_000
    d = scan_inputs(m, n, 2, 4, torch.float32, 0, False, True, False)
    pool = m.normal((n, 2, 4))
    before = pool.clone()
    y = ssm.ssm_state_update_cache(pool, None, d["x"], d["delta"].abs(), d["A"], d["B"], d["C"], D=d["D"])
    dt = d["delta"].abs().double()
    h = torch.exp(dt[:, :, None] * d["A"].double()) * before.double() + (dt * d["x"].double())[:, :, None] * d["B"].double()[:, None, :]
    ref = (h * d["C"].double()[:, None, :]).sum(2) + d["D"].double() * d["x"].double()
    # a few tens of roundings of values below about 30
    assert (pool.double() - h).abs().max() < 64 * 30 * R.U and (y.double() - ref).abs().max() < 64 * 300 * R.U


def test_offsets_beyond_32_bits(ssm):
    """Slots more than 2^31 elements apart (one layer of a large allocation)."""
    dim, n, stride = 40, 16, 1_500_000_000
    store = torch.empty(2 * stride + dim * n, dtype=torch.bfloat16, device="cuda")
    pool = store.as_strided((3, dim, n), (stride, n, 1))
    m = Maker(9)
    ref = m.normal((3, dim, n), torch.bfloat16)
    pool.copy_(ref)
    d = scan_inputs(m, 3, dim, n, torch.bfloat16, 0, True, True, True)
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"], delta_softplus=True)
    args = (d["x"], d["delta"], d["A"], d["B"], d["C"])
    y = ssm.ssm_state_update_cache(pool, i32([2, 0, 1]), *args, **kw)
    y2 = ssm.ssm_state_update_cache(ref, i32([2, 0, 1]), *args, **kw)
    assert torch.equal(y, y2) and torch.equal(pool, ref)
    y = ssm.ssm_scan_packed_fwd(*args, cu_of([2, 1]), cache=pool, cache_slots=i32([2, 1]),
                                has_initial=torch.tensor([True, True], device="cuda"), **kw)
    y2 = ssm.ssm_scan_packed_fwd(*args, cu_of([2, 1]), cache=ref, cache_slots=i32([2, 1]),
                                 has_initial=torch.tensor([True, True], device="cuda"), **kw)
    assert torch.equal(y, y2) and torch.equal(pool, ref)
    codes = torch.zeros(3, dim, n, dtype=torch.int8, device="cuda")
    scales = torch.zeros(3, dim, device="cuda")
    ssm.ssm_cache_store_q8(pool, i32([2]), codes, scales, i32([0]))
    ssm.ssm_cache_load_q8(codes, scales, i32([0]), pool, i32([0]))
    assert (pool[0].float() - ref[2].float()).abs().max() <= scales[0].max() * 0.51 + 0.01


# ---- 8 bits -------------------------------------------------------------------------------------------


def q8_check(ssm, pool, slots, entries, stored, back):
    shape = tuple(pool.shape[1:])
    codes = torch.full((stored,) + shape, 99, dtype=torch.int8, device="cuda")
    scales = torch.full((stored,) + shape[:-1], SENTINEL, device="cuda")
    before = pool.clone()
    ssm.ssm_cache_store_q8(pool, i32(slots), codes, scales, i32(entries))
    assert torch.equal(pool.view(torch.int8), before.view(torch.int8)), "the cache was written"
    q, s = R.quantise(before.float().cpu().numpy())
    want_c, want_s = np.full(codes.shape, 99, np.int64), np.full(scales.shape, SENTINEL, np.float32)
    for a, b in zip(slots, entries):
        if 0 <= a < pool.shape[0] and 0 <= b < stored:
            want_c[b], want_s[b] = q[a], s[a]
    assert np.array_equal(codes.cpu().numpy().astype(np.int64), want_c)
    assert np.array_equal(scales.cpu().numpy(), want_s, equal_nan=True)
    ssm.ssm_cache_load_q8(codes, scales, i32(entries), pool, i32(back))
    want = before.cpu().clone()
    for b, c in zip(entries, back):
        if 0 <= c < pool.shape[0] and 0 <= b < stored:
            val = want_c[b].astype(np.float32) * want_s[b][..., None]
            want[c] = torch.from_numpy(val).to(pool.dtype)
    assert torch.equal(torch.nan_to_num(pool.cpu().float(), nan=7e7), torch.nan_to_num(want.float(), nan=7e7))


@pytest.mark.parametrize("cdtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 4, 8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("rows", [1, 37, 300])
def test_q8_codes_are_the_rounded_quotients(ssm, rows, n, cdtype):
    m = Maker(rows + n)
    pool = m.normal((6, rows, n), DT[cdtype])
    pool *= 10.0 ** torch.linspace(-30, 30, rows, device="cuda")[:, None].to(pool.dtype)
    q8_check(ssm, pool, [4, 0, -1, 5, 6, 2], [1, 3, 0, 9, 2, 0], 4, [0, 1, 2, -1, 3, 5])


def test_q8_borders_and_special_rows(ssm):
    n = 16
    rows = []
    for scale in (1.0, 2.0 ** -60, 3.3e-3, 2.0 ** -130, 2.0 ** -149, 1e36):
        s = np.float32(scale)
        k = np.arange(n, dtype=np.float64)
        for off in (0.5, 0.5 - 1e-7, 0.5 + 1e-7, -0.5):  # on and next to the borders between codes
            v = ((k - 8 + off) * np.float64(s)).astype(np.float32)
            v[0] = np.float32(127.0 * np.float64(s))
            rows.append(v)
    rows.append(np.zeros(n, np.float32))
    rows.append(np.full(n, 1e-45, np.float32))
    rows.append(np.linspace(-1, 1, n).astype(np.float32) * np.float32(190 * 2.0 ** -149))
    rows.append(np.full(n, -3.4028235e38, np.float32))
    for bad in (np.nan, np.inf, -np.inf):
        v = np.linspace(-1, 1, n).astype(np.float32)
        v[5] = bad
        rows.append(v)
    pool = torch.from_numpy(np.stack(rows))[None].repeat(2, 1, 1).cuda()
    q8_check(ssm, pool, [1], [0], 1, [0])


def test_q8_heads_and_fan_out(ssm):
    # a Mamba-2 cache, and one stored prefix read into several slots
    m = Maker(4)
    pool = m.normal((5, 3, 20, 64))
    codes = torch.zeros(2, 3, 20, 64, dtype=torch.int8, device="cuda")
    scales = torch.zeros(2, 3, 20, device="cuda")
    ssm.ssm_cache_store_q8(pool, i32([3]), codes, scales, i32([1]))
    ssm.ssm_cache_load_q8(codes, scales, i32([1, 1, 1]), pool, i32([0, 4, 2]))
    assert torch.equal(pool[0], pool[4]) and torch.equal(pool[0], pool[2])
    off = (pool[0] - pool[3]).abs()
    assert (off <= scales[1][..., None] * (0.5 + 1e-6)).all() and off.max() > 0


# ---- streams, graphs, a run of them together -----------------------------------------------------------


class Layer:
    """One Mamba layer's serving state: the convolution's windows and the scan's states by slot."""

    def __init__(self, m, slots, dim, n, width, dt, cdt):
        self.dim, self.n, self.dt = dim, n, dt
        self.w, self.b = m.normal((dim, width)), m.normal((dim,))
        self.A, self.D, self.bias = m.A(dim, n), m.normal((dim,)), m.normal((dim,)) - 2
        self.windows = torch.full((slots, dim, width - 1), SENTINEL, dtype=dt, device="cuda")
        self.states = torch.full((slots, dim, n), SENTINEL, dtype=cdt, device="cuda")

    def split(self, row):
        d, n = self.dim, self.n
        return dict(x=row[:, :d], z=row[:, d:2 * d], delta=row[:, 2 * d:3 * d], B=row[:, 3 * d:3 * d + n],
                    C=row[:, 3 * d + n:3 * d + 2 * n])

    def width_of_a_row(self):
        return 3 * self.dim + 2 * self.n

    def prompt(self, ssm, rows, cu, slots, initial, longest):
        t = self.split(rows)
        u = ssm.ssm_causal_conv1d_packed_fwd(t["x"], self.w, cu, self.b, cache=self.windows, cache_slots=slots,
                                             has_initial=initial)
        return ssm.ssm_scan_packed_fwd(u, t["delta"], self.A, t["B"], t["C"], cu, D=self.D, z=t["z"],
                                       delta_bias=self.bias, delta_softplus=True, cache=self.states,
                                       cache_slots=slots, has_initial=initial, max_seqlen=longest)

    def step(self, ssm, rows, slots):
        t = self.split(rows)
        u = ssm.ssm_causal_conv1d_update_cache(self.windows, slots, t["x"], self.w, self.b)
        return ssm.ssm_state_update_cache(self.states, slots, u, t["delta"], self.A, t["B"], t["C"], D=self.D,
                                          z=t["z"], delta_bias=self.bias, delta_softplus=True)

    def whole(self, rows):
        """The layer's outputs for a whole sequence in 64 bits, and bounds: the convolution's output is rounded
        to dt between the two operators, which moves the scan's inputs by half a step."""
        t = {k: R.f64(v) for k, v in self.split(rows).items()}
        line = torch.cat([torch.zeros(self.w.shape[1] - 1, self.dim, dtype=torch.float64), t["x"]])
        u, _ = R.conv_rows(line, R.f64(self.w), R.f64(self.b), True)
        y, err, h, eh = R.scan_steps(u, t["delta"], R.f64(self.A), t["B"], t["C"], R.f64(self.D), t["z"],
                                     R.f64(self.bias), True, torch.zeros(self.dim, self.n, dtype=torch.float64))
        # y is linear in u with the coefficients of the same scan: the scan of |u|, |B|, |C|, |D| bounds it
        mag, _, _, _ = R.scan_steps(u.abs(), t["delta"], R.f64(self.A), t["B"].abs(), t["C"].abs(),
                                    R.f64(self.D).abs(), None, R.f64(self.bias), True,
                                    torch.zeros(self.dim, self.n, dtype=torch.float64))
        g = (t["z"] * torch.sigmoid(t["z"])).abs()
        return y, err + mag * g * (R.half_step(self.dt) * 1.01 + 30 * R.U), mag * g


@pytest.mark.parametrize("dtype,cdtype", [("bf16", "f32"), ("f32", "f32")])
def test_prompts_parked_resumed_and_decoded(ssm, dtype, cdtype):
    """Two prompts in chunks, one of them set aside in 8 bits between its chunks, then tokens one by one:
    the sequence that stayed in the cache gives the whole sequence's outputs."""
    m = Maker(21)
    dt = DT[dtype]
    lay = Layer(m, 6, 48, 16, 4, dt, DT[cdtype])
    la, lb, tokens = 90, 61, 6
    ra, rb = (m.normal((n + tokens, lay.width_of_a_row()), dt) for n in (la, lb))
    ya, yb = torch.empty(la + tokens, 48, dtype=dt), torch.empty(lb + tokens, 48, dtype=dt)
    # first chunk: both from zeros, slots 4 and 1
    first = lay.prompt(ssm, torch.cat([ra[:50], rb[:33]]), cu_of([50, 33]), i32([4, 1]), None, 50)
    ya[:50], yb[:33] = first[:50].cpu(), first[50:].cpu()
    # b's state is set aside and comes back in slot 2 (its window is carried over by hand)
    codes = torch.zeros(1, 48, 16, dtype=torch.int8, device="cuda")
    scales = torch.zeros(1, 48, device="cuda")
    kept = lay.states[1].clone()
    ssm.ssm_cache_store_q8(lay.states, i32([1]), codes, scales, i32([0]))
    lay.states[1] = SENTINEL
    ssm.ssm_cache_load_q8(codes, scales, i32([0]), lay.states, i32([2]))
    lay.windows[2] = lay.windows[1]
    moved = (lay.states[2] - kept).abs().cpu().double()
    assert (moved <= scales[0][:, None].cpu().double() * 0.5000001 + 1e-12).all()
    # second chunk: both go on from their slots, packed the other way round, one padded sequence
    init = torch.tensor([True, True, True], device="cuda")
    second = lay.prompt(ssm, torch.cat([rb[33:lb], ra[50:la]]), cu_of([lb - 33, la - 50, 0]), i32([2, 4, -1]), init, 40)
    yb[33:lb], ya[50:la] = second[:lb - 33].cpu(), second[lb - 33:].cpu()
    for k in range(tokens):
        rows = torch.stack([ra[la + k], torch.zeros_like(ra[0]), rb[lb + k]])
        out = lay.step(ssm, rows, i32([4, -1, 2])).cpu()
        ya[la + k], yb[lb + k] = out[0], out[2]
    ref, err, _ = lay.whole(ra)
    R.check(ya, ref, err, dt, "the sequence in the cache")
    ref, err, mag = lay.whole(rb)
    R.check(yb[:33], ref[:33], err[:33], dt, "the other before it was set aside")
    # 8 bits move each state by at most half a scale (1 / 254 of the row's largest), which decays from there
    t = {k: R.f64(v) for k, v in lay.split(rb).items()}
    drift, _, _, _ = R.scan_steps(torch.zeros(lb + tokens - 33, 48, dtype=torch.float64), t["delta"][33:], R.f64(lay.A),
                                  t["B"][33:], t["C"][33:].abs(), None, None, R.f64(lay.bias), True, moved)
    g = (t["z"] * torch.sigmoid(t["z"])).abs()[33:]
    R.check(yb[33:], ref[33:], err[33:] + drift * g * 1.01, dt, "the other afterwards")


def serving_round(ssm, lay, rows, cu, slots, init, tok, tslots, codes, scales, where, outs, longest):
    outs[0].copy_(lay.prompt(ssm, rows, cu, slots, init, longest))
    outs[1].copy_(lay.step(ssm, tok, tslots))
    ssm.ssm_cache_store_q8(lay.states, slots, codes, scales, where)
    ssm.ssm_cache_load_q8(codes, scales, where, lay.states, tslots)


@pytest.mark.parametrize("how", ["graph", "stream"])
def test_captured_and_on_another_stream(ssm, how):
    m = Maker(33)
    dt = torch.bfloat16
    lay = Layer(m, 8, 64, 16, 4, dt, torch.float32)
    lens = [600, 7, 40]  # the first is cut into pieces where the rule says so: workspace in the graph
    rows = m.normal((sum(lens), lay.width_of_a_row()), dt)
    tok = m.normal((3, lay.width_of_a_row()), dt)
    cu, slots, tslots, where = cu_of(lens), i32([5, 0, 3]), i32([0, -1, 5]), i32([2, 0, 1])
    init = torch.tensor([True, False, True], device="cuda")
    codes = torch.zeros(3, 64, 16, dtype=torch.int8, device="cuda")
    scales = torch.zeros(3, 64, device="cuda")
    w0, s0 = m.normal(lay.windows.shape, dt), m.normal(lay.states.shape)
    state = [lay.windows, lay.states, codes, scales]

    def reset():
        lay.windows.copy_(w0)
        lay.states.copy_(s0)
        codes.zero_()
        scales.zero_()

    def make_outs():
        return [torch.zeros(sum(lens), 64, dtype=dt, device="cuda"), torch.zeros(3, 64, dtype=dt, device="cuda")]

    args = (rows, cu, slots, init, tok, tslots, codes, scales, where)
    live = [0, 2]  # rows of the step that have a slot
    reset()
    eager = make_outs()
    serving_round(ssm, lay, *args, eager, 600)
    torch.cuda.synchronize()
    want = [t.clone() for t in state] + [eager[0].clone(), eager[1][live].clone()]
    outs = make_outs()
    side = torch.cuda.Stream()
    if how == "graph":
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            serving_round(ssm, lay, *args, outs, 600)
    for rep in range(4):
        reset()
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        if how == "graph":
            g.replay()
        else:
            with torch.cuda.stream(side):
                serving_round(ssm, lay, *args, outs, 600)
        torch.cuda.synchronize()
        got = [t.clone() for t in state] + [outs[0].clone(), outs[1][live].clone()]
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"repeat {rep} differs"
        reset()
        serving_round(ssm, lay, *args, make_outs(), 600)  # eager work between the replays
        torch.cuda.synchronize()
        say(f"  {how} {rep} matches eager")


def test_given_stream(ssm):
    m = Maker(41)
    d = scan_inputs(m, 900, 32, 16, torch.bfloat16, 0, True, True, True)
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"], delta_softplus=True, max_seqlen=900)
    args = (d["x"], d["delta"], d["A"], d["B"], d["C"], cu_of([900]))
    want = ssm.ssm_scan_packed_fwd(*args, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream, 0):
        got = ssm.ssm_scan_packed_fwd(*args, stream=s, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_no_rows_no_sequences(ssm):
    z = torch.zeros
    pool = torch.ones(2, 8, 16, device="cuda")
    A = -torch.ones(8, 16, device="cuda")
    e = z(0, 8, device="cuda")
    y = ssm.ssm_scan_packed_fwd(e, e, A, z(0, 16, device="cuda"), z(0, 16, device="cuda"), i32([0, 0, 0]), cache=pool)
    assert y.shape == (0, 8) and (pool == 1).all()
    y = ssm.ssm_state_update_cache(pool, i32([]), e, e, A, z(0, 16, device="cuda"), z(0, 16, device="cuda"))
    assert y.shape == (0, 8) and (pool == 1).all()
    x = z(3, 8, device="cuda")
    y0 = torch.full((3, 8), SENTINEL, device="cuda")
    ssm.ssm_causal_conv1d_packed_fwd(x, z(8, 4, device="cuda"), i32([0]), y=y0)
    assert (y0 == SENTINEL).all()


@pytest.mark.parametrize("nseq", [63, 64, 65, 300, 5000])
def test_conv_packed_finds_every_sequence(ssm, nseq):
    # the search for a tile's first sequence: 64 probes a round; empty sequences among them
    lens = [(i * 7) % 5 for i in range(nseq)]
    total, dim = sum(lens), 8
    m = Maker(nseq)
    x, w = m.normal((total, dim)), m.normal((dim, 4))
    pool = m.normal((nseq, dim, 3))
    before = pool.clone()
    y = ssm.ssm_causal_conv1d_packed_fwd(x, w, cu_of(lens), None, False, cache=pool,
                                         has_initial=torch.ones(nseq, dtype=torch.bool, device="cuda"))
    lines, out = [], []
    r0 = 0
    for i, L in enumerate(lens):
        line = torch.cat([R.f64(before[i]).T, R.f64(x[r0:r0 + L])])
        out.append(R.conv_rows(line, R.f64(w), None, False))
        lines.append(line[line.shape[0] - 3:].T.float())
        r0 += L
    R.check(y, torch.cat([o[0] for o in out]), torch.cat([o[1] for o in out]), torch.float32, f"{nseq} sequences")
    assert torch.equal(pool.cpu(), torch.stack(lines))


def test_scan_packed_infinite_input_and_padding_states(ssm):
    # dstate 1 and 2 are computed as 4: an infinite input gives the infinities of the formula, not NaN
    for n in (1, 2):
        x = torch.zeros(6, 20, device="cuda")
        x[2] = float("inf")
        one = torch.ones(6, n, device="cuda")
        y = ssm.ssm_scan_packed_fwd(x, torch.ones_like(x), -torch.ones(20, n, device="cuda"), one, one, cu_of([6]))
        assert (y[:2] == 0).all() and torch.isinf(y[2:]).all()
