"""The gated recurrence on the GPU against its 64-bit form (gated_ref.py), element by element within
bounds that count roundings: batches forward and backward, packed prompts, single tokens."""
import itertools

import pytest
import torch

import gated_ref as R
import selective_state_space_61_amd as ssm
from gpu_util import say

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssm.load_library()


def make(shape, dtype, seed, z=True, bias=True, wide=False):
    """x, the gates and z in this dtype (columns of one wider tensor if wide), parameters, on the GPU."""
    g = torch.Generator().manual_seed(seed)
    dim = shape[-1]
    if wide:
        whole = torch.randn(shape[:-1] + (4 * dim + 3,), generator=g).to(dtype).cuda()
        cols = [whole[..., k * dim:(k + 1) * dim] for k in range(4)]
    else:
        cols = [torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(4)]
    t = dict(zip(("x", "a_gate", "x_gate", "z"), cols))
    if not z:
        t["z"] = None
    # decays of an open gate from 0.2 to 0.9999
    t["a_param"] = (torch.rand(dim, generator=g) * 10 - 11).cuda()
    t["a_bias"], t["x_bias"] = (torch.randn(dim, generator=g).cuda() if bias else None for _ in range(2))
    return t


def host(t):
    """The reference's arguments, rows first."""
    names = dict(x="x", a_gate="ag", x_gate="xg", a_param="param", a_bias="ab", x_bias="xb", z="z")
    d = {names[k]: R.f64(v) for k, v in t.items()}
    for k in ("x", "ag", "xg", "z"):
        if d[k] is not None and d[k].dim() == 3:
            d[k] = d[k].transpose(0, 1)
    return d


SHAPES = [(1, 1, 1), (2, 3, 1), (1, 2, 2), (2, 7, 3), (1, 1, 64), (3, 64, 64), (2, 65, 130), (1, 127, 66), (4, 129, 63),
          (5, 31, 257), (1, 700, 100), (40, 5, 20), (2, 1030, 68), (130, 1, 72), (3, 256, 40), (2, 255, 33), (7, 257, 129), (2, 4096, 5)]


@pytest.mark.parametrize("shape,dtype,z,states", [(s, d, (k + n) % 3 != 0, (k + n) % 2 == 0)
                                                  for n, s in enumerate(SHAPES) for k, d in enumerate((BF, F))])
def test_batches(shape, dtype, z, states):
    batch, seqlen, dim = shape
    say(f"[case] gated batch {shape} {dtype} z={z} states={states}")
    t = make(shape, dtype, seqlen + dim, z=z, bias=states or z)
    g = torch.Generator().manual_seed(5)
    h0, dlast = (torch.randn(batch, dim, generator=g).cuda() if states else None for _ in range(2))
    dy = torch.randn(shape, generator=g).to(dtype).cuda()
    y, last, saved = ssm.ssm_gated_scan_fwd_ckpt(**t, initial_state=h0)
    grads = ssm.ssm_gated_scan_bwd_ckpt(dy=dy, checkpoints=saved, initial_state=h0, dlast_state=dlast, **t)
    again, again_last = ssm.ssm_gated_scan_fwd(**t, initial_state=h0)
    torch.cuda.synchronize()
    assert torch.equal(y, again) and torch.equal(last, again_last)
    d = host(t)
    yr, ey, h, eh = R.forward(**d, h0=R.f64(h0))
    R.check(y, yr.transpose(0, 1), ey.transpose(0, 1), dtype, "y")
    R.check(last, h[-1], eh[-1], F, "last_state")
    assert saved.shape == ssm.gated_checkpoint_shape(batch, seqlen, dim)
    if batch > 1 and seqlen >= 256:
        rows, erows = (v[63::64].transpose(0, 1).reshape(-1, dim) for v in (h, eh))
    else:
        rows, erows = (v.transpose(0, 1).reshape(batch * seqlen, dim)[63::64] for v in (h, eh))
    R.check(saved, rows, erows, F, "checkpoints")
    ref = R.backward(**d, dy=R.f64(dy).transpose(0, 1), h0=R.f64(h0), dlast=R.f64(dlast))
    for k, v in grads.items():
        if v is None:
            assert {"dz": t["z"], "da_bias": t["a_bias"], "dx_bias": t["x_bias"], "dinitial_state": h0}[k] is None
            continue
        val, ev = ref[k]
        if val.dim() == 3:
            val, ev = val.transpose(0, 1), ev.transpose(0, 1)
        R.check(v, val, ev, v.dtype, k)


@pytest.mark.parametrize("shape", [(9, 40, 70), (11, 41, 33), (50, 2, 64), (13, 20, 130), (3, 128, 65), (3, 64, 66), (200, 31, 5),
                                   (70, 7, 3), (33, 11, 1), (9, 32, 2)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_batches_of_short_sequences(shape, dtype):
    """Several whole sequences in a tile, forward, backward or both; the forward's checkpoints then lie anywhere in
    its tiles."""
    test_batches(shape, dtype, True, True)
    batch, seqlen, dim = shape
    t = make(shape, dtype, 7)
    y, last, saved = ssm.ssm_gated_scan_fwd_ckpt(**dict(t, z=None))
    rows = torch.arange(63, batch * seqlen, 64)
    d = host(dict(t, z=None))
    _, _, h, eh = R.forward(**d)
    R.check(saved, h.transpose(0, 1).reshape(-1, dim)[rows], eh.transpose(0, 1).reshape(-1, dim)[rows], F, "checkpoints")


@pytest.mark.parametrize("dtype", [BF, F])
def test_a_long_sequence(dtype):
    """Hundreds of tiles handing states on, forward and backward."""
    t = make((1, 20011, 12), dtype, 3)
    t["a_param"] = t["a_param"] - 4  # decays to 1e-6: the states of far tiles matter
    dy = torch.randn(1, 20011, 12, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()
    y, last, saved = ssm.ssm_gated_scan_fwd_ckpt(**t)
    grads = ssm.ssm_gated_scan_bwd_ckpt(dy=dy, checkpoints=saved, **t)
    d = host(t)
    yr, ey, h, eh = R.forward(**d)
    R.check(y, yr.transpose(0, 1), ey.transpose(0, 1), dtype, "y")
    R.check(last, h[-1], eh[-1], F, "last_state")
    ref = R.backward(**d, dy=R.f64(dy).transpose(0, 1))
    for k, v in grads.items():
        if v is not None:
            val, ev = ref[k]
            R.check(v, *((val.transpose(0, 1), ev.transpose(0, 1)) if val.dim() == 3 else (val, ev)), v.dtype, k)


def test_results_do_not_depend_on_timing():
    """Bit for bit the same beside other work on another stream, forward and backward."""
    t = make((4, 3000, 320), BF, 8)
    dy = torch.randn(4, 3000, 320, generator=torch.Generator().manual_seed(6)).to(BF).cuda()
    run = lambda: (lambda f: (*f, *ssm.ssm_gated_scan_bwd_ckpt(dy=dy, checkpoints=f[2], **t).values()))(  # noqa: E731
        ssm.ssm_gated_scan_fwd_ckpt(**t))
    ref = [v for v in run() if v is not None]
    side, load = torch.cuda.Stream(), torch.randn(2000, 2000, device="cuda")
    for rep in range(6):
        with torch.cuda.stream(side):
            for _ in range(rep):
                load = (load @ load).clamp(-1, 1)
        got = [v for v in run() if v is not None]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), f"run {rep}"


def packed(lens, lead=0, tail=0):
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32).cuda(), cu, cu[-1] + tail


LENS = [[1], [2, 1, 1], [5, 0, 40, 1, 200, 0, 0, 3], [300], [128, 128, 64], [127, 1, 129, 0, 255], [1] * 150, [0, 0, 7],
        [64] * 5]


@pytest.mark.parametrize("n,dtype,cdtype,dim", [(n, d, c, m) for n, (d, c, m) in itertools.product(
    range(len(LENS)), [(BF, F, 72), (F, BF, 33), (BF, BF, 3), (F, F, 130)])])
def test_packed(n, dtype, cdtype, dim):
    lens = LENS[n]
    say(f"[case] gated packed {lens[:8]} dim={dim} {dtype} cache {cdtype}")
    cu, starts, total = packed(lens, lead=n % 3, tail=(n % 2) * 5)
    nseq = len(lens)
    g = torch.Generator().manual_seed(n)
    t = make((total, dim), dtype, 10 + n, z=n % 2 == 0, wide=n % 3 == 1)
    wide_y = torch.full((total, dim + 5), 7.0, dtype=dtype, device="cuda")
    y = wide_y[:, 2:2 + dim]
    cache = torch.randn(nseq + 2, 2, dim, generator=g).to(cdtype).cuda()[:, 1]  # one layer of an allocation
    before = cache.clone()
    slots = torch.randperm(nseq + 2, generator=g)[:nseq].int()
    if nseq > 2:
        slots[1] = -1
    if nseq > 4:
        slots[2] = nseq + 2
    init = torch.rand(nseq, generator=g) < 0.6
    out = ssm.ssm_gated_scan_packed_fwd(**t, cu_seqlens=cu, cache=cache, cache_slots=slots.cuda(), has_initial=init.cuda(), y=y)
    torch.cuda.synchronize()
    assert out.data_ptr() == y.data_ptr()
    d = host(t)
    touched = set()
    for s, slot in enumerate(slots.tolist()):
        a, b = starts[s], starts[s + 1]
        real = 0 <= slot < nseq + 2
        h0 = R.f64(before[slot]) if real and init[s] else torch.zeros(dim, dtype=torch.float64)
        rows = {k: (v[a:b] if k in ("x", "ag", "xg", "z") and v is not None else v) for k, v in d.items()}
        yr, ey, h, eh = R.forward(**rows, h0=h0)
        R.check(y[a:b], yr, ey, dtype, f"y of sequence {s}")
        if real and b > a:
            touched.add(slot)
            R.check(cache[slot], h[-1], eh[-1], cdtype, f"state of sequence {s}")
    for slot in range(nseq + 2):
        if slot not in touched:
            assert torch.equal(cache[slot], before[slot])
    # rows of no sequence, and what lies beside the rows
    rest = torch.ones(total, dtype=torch.bool)
    rest[starts[0]:starts[-1]] = False
    assert (wide_y[rest.cuda()] == 7).all() and (wide_y[:, :2] == 7).all() and (wide_y[:, 2 + dim:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F])
def test_one_row_of_a_large_projection(dtype):
    """The last row of a long text's projections: its distance to the next row, which is not there, does not matter."""
    dim, g = 72, torch.Generator().manual_seed(1)
    whole = torch.randn((1, 2048, 5120), generator=g).to(dtype).cuda()
    last = whole[:, -1]
    cols = {k: last[:, n * dim:(n + 1) * dim] for n, k in enumerate(("x", "a_gate", "x_gate", "z"))}
    assert cols["x"].stride(0) > 2 ** 23
    param, cache = torch.full((dim,), -4.0).cuda(), torch.randn(1, dim, generator=g).cuda()
    y = torch.empty((1, 2048, 5120), dtype=dtype, device="cuda")[:, -1, 8:8 + dim]
    before, yes = cache.clone(), torch.ones(1, dtype=torch.bool).cuda()
    ssm.ssm_gated_scan_packed_fwd(**cols, a_param=param, cu_seqlens=packed([1])[0], cache=cache, has_initial=yes, y=y)
    yr, ey, h, eh = R.forward(**host(dict(cols, a_param=param, a_bias=None, x_bias=None)), h0=R.f64(before[0]))
    R.check(y, yr, ey, dtype, "y")
    R.check(cache[0], h[-1], eh[-1], F, "state")


def test_packed_without_a_cache_is_the_batch():
    """Equal lengths packed are the rows of a batch: the same tiles, the same bits."""
    t = make((6, 90, 100), BF, 4)
    y, _ = ssm.ssm_gated_scan_fwd(**t)
    rows = {k: (v.reshape(540, 100) if k in ("x", "a_gate", "x_gate", "z") else v) for k, v in t.items()}
    cu = torch.arange(0, 541, 90, dtype=torch.int32).cuda()
    assert torch.equal(ssm.ssm_gated_scan_packed_fwd(**rows, cu_seqlens=cu), y.view(540, 100))


@pytest.mark.parametrize("dtype", [BF, F])
def test_values_of_one_sequence_never_reach_another(dtype):
    """NaN and infinities in x, a gate, z and a cached state: only their own sequence's rows show them."""
    lens = [40, 130, 7, 300, 64, 1, 90]
    cu, starts, total = packed(lens)
    bad = [1, 3, 5]
    for k, value in itertools.product(("x", "a_gate", "x_gate", "z", "cache"), (float("nan"), float("inf"), float("-inf"))):
        t = make((total, 70), dtype, 2)
        cache = torch.randn(7, 70, generator=torch.Generator().manual_seed(3)).cuda()
        ones = torch.ones(7, dtype=torch.bool).cuda()
        clean_cache = cache.clone()
        clean = ssm.ssm_gated_scan_packed_fwd(**t, cu_seqlens=cu, cache=clean_cache, has_initial=ones)
        for s in bad:
            if k == "cache":
                cache[s] = value
            else:
                t[k][starts[s]:starts[s + 1]][-1] = value
        y = ssm.ssm_gated_scan_packed_fwd(**t, cu_seqlens=cu, cache=cache, has_initial=ones)
        for s in range(7):
            if s not in bad:
                assert torch.equal(y[starts[s]:starts[s + 1]], clean[starts[s]:starts[s + 1]]), (k, value, s)
                assert torch.equal(cache[s], clean_cache[s]), (k, value, s)


@pytest.mark.parametrize("dtype", [BF, F])
def test_gradients_of_one_sequence_never_reach_another(dtype):
    for k, value in itertools.product(("x", "a_gate", "z", "dy"), (float("nan"), float("inf"))):
        t = dict(make((5, 50, 70), dtype, 2), dy=torch.ones(5, 50, 70, dtype=dtype).cuda())
        run = lambda: ssm.ssm_gated_scan_bwd_ckpt(checkpoints=ssm.ssm_gated_scan_fwd_ckpt(  # noqa: E731
            **{n: v for n, v in t.items() if n != "dy"})[2], **t)
        clean = run()
        t[k] = t[k].clone()
        t[k][1, 20] = value
        t[k][3] = value
        got = run()
        for name in ("dx", "da_gate", "dx_gate", "dz"):
            for b in (0, 2, 4):
                assert torch.equal(got[name][b], clean[name][b]), (k, value, name, b)


def test_closed_gates_and_extreme_parameters():
    """a_gate of -inf keeps the state and takes no input; +inf and huge parameters forget it; gradients are
    finite, and those through a closed gate 0."""
    t = make((2, 150, 64), F, 1, bias=False)
    t["a_gate"][:, 10:20] = float("-inf")
    t["a_gate"][:, 30] = float("inf")
    t["a_gate"][:, 40:50] = -100.0
    t["x_gate"][:, 60] = float("-inf")
    t["x_gate"][:, 61] = float("inf")
    t["a_param"][:8] = 1e30
    t["a_param"][8:16] = -120.0
    t["a_param"][16:20] = float("-inf")
    dy = torch.randn(2, 150, 64, generator=torch.Generator().manual_seed(6)).cuda()
    h0 = torch.randn(2, 64, generator=torch.Generator().manual_seed(7)).cuda()
    plain = dict(t, z=None)
    y, last, saved = ssm.ssm_gated_scan_fwd_ckpt(**plain, initial_state=h0)
    grads = ssm.ssm_gated_scan_bwd_ckpt(**plain, dy=dy, checkpoints=saved, initial_state=h0)
    assert torch.isfinite(y).all()
    assert torch.equal(y[:, :, 16:20], h0[:, None, 16:20].expand(-1, 150, -1))
    for k, v in grads.items():
        if v is not None:
            assert torch.isfinite(v).all(), k
    assert (grads["da_gate"][:, 10:20] == 0).all() and (grads["dx"][:, 10:20] == 0).all()
    d = host(plain)
    yr, ey, h, eh = R.forward(**d, h0=R.f64(h0))
    ok = torch.ones(64, dtype=torch.bool)
    ok[:8] = False  # (l is -1e30 there in place of -8e30: a is 0 either way)
    R.check(y[:, :, 8:], yr.transpose(0, 1)[:, :, ok], ey.transpose(0, 1)[:, :, ok], F, "y")
    # rows whose exact values are equal: each is off by its bound at most, so two differ by the sum of theirs
    # (not bit for bit: the composed map of a part's rows rounds otherwise than the rows one by one)
    yc, ec = y.cpu().double().transpose(0, 1)[:, :, ok], (ey + yr.abs() * R.U)[:, :, ok]
    assert ((yc[10:20] - yc[9]).abs() <= ec[10:20] + ec[9]).all()


@pytest.mark.parametrize("dtype", [BF, F])
def test_huge_inputs_behind_closed_gates(dtype):
    """Inputs up to the type's largest that a closed gate keeps out leave no trace in states and gradients."""
    t = make((2, 150, 66), dtype, 3)
    t["a_gate"][:, 20:90] = float("-inf")
    plain = dict(t, x=torch.where(t["a_gate"].isinf(), torch.zeros_like(t["x"]), t["x"]))
    t["x"] = torch.where(t["a_gate"].isinf(), t["x"].sign() * torch.finfo(dtype).max, t["x"])
    dy = torch.randn(2, 150, 66, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()
    got, want = [], []
    for out, d in ((got, t), (want, plain)):
        y, last, saved = ssm.ssm_gated_scan_fwd_ckpt(**d)
        out += [y, last, *(v for v in ssm.ssm_gated_scan_bwd_ckpt(**d, dy=dy, checkpoints=saved).values() if v is not None)]
    for a, b in zip(got, want):
        assert torch.isfinite(b).all() and torch.equal(a, b)


def test_a_parameter_that_is_no_number():
    """NaN in a_param is NaN in its channel's rows, states and gradients, and in no other's."""
    for shape in ((2, 70, 130), (300, 1, 5)):
        t = make(shape, BF, 4)
        bad = dict(t, a_param=t["a_param"].clone())
        bad["a_param"][3] = float("nan")
        other = torch.arange(shape[-1]) != 3
        dy = torch.ones(shape, dtype=BF, device="cuda")
        outs = []
        for d in (t, bad):
            y, last, saved = ssm.ssm_gated_scan_fwd_ckpt(**d)
            grads = ssm.ssm_gated_scan_bwd_ckpt(**d, dy=dy, checkpoints=saved)
            cache = torch.ones(shape[0], shape[-1], device="cuda")
            rows = {k: (v[:, 0].contiguous() if k in ("x", "a_gate", "x_gate", "z") else v) for k, v in d.items()}
            outs.append([y, last, grads["dx"], grads["da_param"], ssm.ssm_gated_update_cache(cache, None, **rows), cache])
        for clean, got in zip(*outs):
            assert torch.equal(clean[..., other], got[..., other])
            assert got[..., 3].isnan().all()


def infinite_case(batch, rows, dim, dtype, seed, z=False):
    """Channels whose decays of one step run from 0.99 to e^-85 (fp32's least normal number is e^-87.3): no step's is
    0 in fp32, that of most stretches is.  All gates near 0.5 to 1, x of either sign."""
    t = make((batch, rows, dim), dtype, seed, z=z, bias=False)
    t["a_gate"], t["x_gate"] = t["a_gate"].abs(), t["x_gate"].abs()
    rate = torch.logspace(-2, 1.02, dim, dtype=torch.float64)  # softplus(a_param): at most 10.5, times 8 at most 84
    t["a_param"] = torch.log(torch.expm1(rate)).float().cuda()
    return t


def kinds(v):
    """Each value's kind: finite 0, +inf 1, -inf 2, NaN 3."""
    return (v == float("inf")).int() + 2 * (v == float("-inf")).int() + 3 * v.isnan().int()


@pytest.mark.parametrize("batch,rows,dim", [(1, 700, 70), (3, 700, 65), (5, 40, 70), (3, 90, 70), (1, 1400, 5), (2, 300, 3), (2, 300, 1)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_an_infinite_state_stays(batch, rows, dim, dtype):
    """A state that has become infinite (by an input or from the start) stays so in batches, packed prompts and their
    states, wherever stretches and tiles begin, as it does token by token; and so does an infinite adjoint."""
    say(f"[case] gated infinite {batch} x {rows} x {dim} {dtype}")
    t = infinite_case(batch, rows, dim, dtype, dim)
    for at, sign in ((3, 1.0), (rows // 2, -1.0), (-1, 1.0)):
        x = t["x"].clone()
        h0 = torch.zeros(batch, dim, device="cuda")
        if at < 0:
            h0[0] = sign * INF
        else:
            x[0, at] = sign * INF
        d = dict(t, x=x)
        y, last, saved = ssm.ssm_gated_scan_fwd_ckpt(**d, initial_state=h0)
        want = torch.zeros(batch, rows, dim, dtype=torch.int32, device="cuda")
        want[0, max(at, 0):] = 1 if sign > 0 else 2
        assert torch.equal(kinds(y), want) and torch.equal(kinds(last), want[:, -1]), at
        kept = want[:, 63::64].reshape(-1, dim) if batch > 1 and rows >= 256 else want.view(-1, dim)[63::64]
        assert torch.equal(kinds(saved), kept), at
        flat = {k: (v.view(batch * rows, dim) if v is not None and v.dim() == 3 else v) for k, v in d.items()}
        cu = torch.arange(0, batch * rows + 1, rows, dtype=torch.int32).cuda()
        cache = h0.clone()
        yp = ssm.ssm_gated_scan_packed_fwd(**flat, cu_seqlens=cu, cache=cache, has_initial=torch.ones(batch, dtype=torch.bool).cuda())
        assert torch.equal(kinds(yp), want.view(-1, dim)) and torch.equal(kinds(cache), want[:, -1]), at
        # the states that the backward works out again: dz is dy h silu'(z)
        z, dy = torch.ones_like(x), torch.ones_like(x)
        dz = ssm.ssm_gated_scan_bwd_ckpt(**dict(d, z=z), dy=dy, checkpoints=saved, initial_state=h0)["dz"]
        assert torch.equal(kinds(dz), want), at
        # an infinite gradient of the last state, or of a row
        dlast = torch.zeros(batch, dim, device="cuda")
        if at < 0:
            dlast[0] = sign * INF
        else:
            dy[0, at] = sign * INF
        fwd = ssm.ssm_gated_scan_fwd_ckpt(**t)
        got = ssm.ssm_gated_scan_bwd_ckpt(**t, dy=dy, checkpoints=fwd[2], dlast_state=dlast, initial_state=torch.zeros_like(dlast))
        want.zero_()
        want[0, :at + 1 if at >= 0 else rows] = 1 if sign > 0 else 2
        assert torch.equal(kinds(got["dx"]), want) and torch.equal(kinds(got["dinitial_state"]), want[:, 0]), at


@pytest.mark.parametrize("dtype", [BF, F])
def test_an_infinite_state_meets_a_step_without_decay_left(dtype):
    """A step whose decay is 0 in fp32 makes an infinite state NaN, in a prompt at the same row as token by token,
    whatever stretch or tile that row lies in; a finite state is forgotten."""
    rows, dim, start = 420, 66, 50
    for at in (51, 64, 130, 383):
        t = infinite_case(1, rows, dim, dtype, at)
        t["x"][0, start, ::2] = INF
        t["a_gate"][0, at, ::3] = INF  # a rate of 1e3 on top of it: every such step's decay is 0
        t["a_param"][::3] = 125.0
        t["a_gate"][0, :, ::3][t["a_gate"][0, :, ::3] != INF] = -5.0  # (of 6.7 elsewhere: e^-6.7)
        flat = {k: (v[0] if v is not None and v.dim() == 3 else v) for k, v in t.items()}
        cu, cache = packed([rows])[0], torch.zeros(1, dim).cuda()
        y = ssm.ssm_gated_scan_packed_fwd(**flat, cu_seqlens=cu, cache=cache)
        alone = torch.zeros(1, dim).cuda()
        ys = [ssm.ssm_gated_update_cache(alone, None, **{k: (v[n:n + 1] if v is not None and v.dim() == 2 else v)
                                                         for k, v in flat.items()}) for n in range(rows)]
        assert torch.equal(kinds(y), kinds(torch.cat(ys))) and torch.equal(kinds(cache), kinds(alone)), at
        k = kinds(y)
        assert (k[start:, 2::6] == 1).all() and (k[start:at, ::6] == 1).all() and (k[at:, ::6] == 3).all() and (k[:, 1::2] == 0).all()


@pytest.mark.parametrize("dim,dtype,cdtype", [(66, BF, F), (65, BF, BF), (67, BF, F), (65, F, BF), (129, BF, BF), (194, BF, F)])
def test_packed_with_a_short_last_block(dim, dtype, cdtype):
    """Channels past a multiple of 64 that fill no lane: each state is read and written by one workgroup alone,
    also where the cache is updated in place; twice as many short sequences begin in a tile as it has rows."""
    lens = [1, 0, 0, 2, 0] * 60 + [200, 1]
    cu, starts, total = packed(lens)
    g = torch.Generator().manual_seed(dim)
    t = make((total, dim), dtype, dim)
    cache = torch.randn(len(lens), dim, generator=g).to(cdtype).cuda()
    before = cache.clone()
    init = torch.ones(len(lens), dtype=torch.bool).cuda()
    y = ssm.ssm_gated_scan_packed_fwd(**t, cu_seqlens=cu, cache=cache, has_initial=init)
    d = host(t)
    for s, n in enumerate(lens):
        a, b = starts[s], starts[s + 1]
        if n == 0:
            assert torch.equal(cache[s], before[s])
            continue
        rows = {k: (v[a:b] if k in ("x", "ag", "xg", "z") else v) for k, v in d.items()}
        yr, ey, h, eh = R.forward(**rows, h0=R.f64(before[s]))
        R.check(y[a:b], yr, ey, dtype, f"y of sequence {s}")
        R.check(cache[s], h[-1], eh[-1], cdtype, f"state of sequence {s}")


def test_no_decay_at_all():
    """a_scale 0: the states never move."""
    t = make((2, 200, 10), BF, 1)
    h0 = torch.randn(2, 10).cuda()
    y, last = ssm.ssm_gated_scan_fwd(**dict(t, z=None), a_scale=0.0, initial_state=h0)
    assert torch.equal(last, h0) and torch.equal(y, h0[:, None].expand(-1, 200, -1).to(BF))


@pytest.mark.parametrize("batch,dim,dtype,cdtype,wide", [(1, 1, BF, F, False), (1, 64, F, F, False), (3, 3, F, BF, True),
                                                         (2, 5, BF, BF, True), (7, 1536, BF, F, True), (250, 130, BF, BF, True),
                                                         (1030, 1030, F, F, False), (9, 5119, F, BF, True)])
def test_steps(batch, dim, dtype, cdtype, wide):
    say(f"[case] gated step {batch} x {dim} {dtype} {cdtype}")
    t = make((batch, dim), dtype, batch + dim, z=dim % 2 == 1, wide=wide)
    g = torch.Generator().manual_seed(1)
    slots = torch.randperm(batch + 3, generator=g)[:batch].int()
    if batch > 2:
        slots[1], slots[2] = -1, batch + 3
    cache = torch.randn(batch + 3, 3, dim, generator=g).to(cdtype).cuda()[:, 2]
    before = cache.clone()
    y = torch.full((batch, dim), 7.0, dtype=dtype, device="cuda")
    ssm.ssm_gated_update_cache(cache, slots.cuda(), y=y, **t)
    torch.cuda.synchronize()
    on = ((slots >= 0) & (slots < batch + 3)).nonzero()[:, 0]
    d = {k: (v[on] if v is not None and v.dim() == 2 else v) for k, v in host(t).items()}
    pick = slots[on].long()
    one = {k: (v[None] if v is not None and v.dim() == 2 else v) for k, v in d.items()}
    yr, ey, h, eh = R.forward(**one, h0=R.f64(before)[pick])
    R.check(y[on.cuda()], yr[0], ey[0], dtype, "y")
    R.check(cache[pick.cuda()], h[0], eh[0], cdtype, "state")
    off = torch.ones(batch + 3, dtype=torch.bool)
    off[pick] = False
    assert torch.equal(cache[off.cuda()], before[off.cuda()])
    if batch > 2:
        assert (y[1:3] == 7).all()


def test_steps_continue_a_prompt():
    """A prompt in one call, in two, and its last tokens one by one: the same states within their bounds."""
    dim = 100
    t = make((90, dim), F, 9)
    d = host(t)
    rows = lambda a, b: {k: (v[a:b] if v is not None and v.dim() == 2 else v) for k, v in t.items()}  # noqa: E731
    yr, ey, h, eh = R.forward(**d)
    slot, yes = torch.tensor([1], dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.bool).cuda()
    for cut, cut2 in ((30, 90), (64, 64), (1, 60)):
        cache = torch.full((3, dim), 5.0).cuda()
        ys = [ssm.ssm_gated_scan_packed_fwd(**rows(0, cut), cu_seqlens=packed([cut])[0], cache=cache, cache_slots=slot)]
        if cut2 > cut:
            ys.append(ssm.ssm_gated_scan_packed_fwd(**rows(cut, cut2), cu_seqlens=packed([cut2 - cut])[0], cache=cache,
                                                    cache_slots=slot, has_initial=yes))
        ys += [ssm.ssm_gated_update_cache(cache, slot, **rows(k, k + 1)) for k in range(cut2, 90)]
        R.check(torch.cat(ys), yr, ey, F, f"y, cut at {cut} and {cut2}")
        R.check(cache[1], h[-1], eh[-1], F, "state")
        assert (cache[::2] == 5).all()


def test_captured_into_graphs():
    """Forward, backward, packed and step captured; every replay gives the eager call's bits, with other work
    between the replays."""
    t = make((3, 400, 96), BF, 21)
    dy = torch.randn(3, 400, 96, generator=torch.Generator().manual_seed(6)).to(BF).cuda()
    rows = {k: (v.reshape(1200, 96) if v is not None and v.dim() == 3 else v) for k, v in t.items()}
    one = {k: (v[:5, 0] if v is not None and v.dim() == 3 else v) for k, v in make((5, 1, 96), BF, 22).items()}
    one = {k: (v.contiguous() if v is not None else v) for k, v in one.items()}
    cu = packed([700, 1, 499])[0]
    start = torch.randn(8, 96).cuda()

    def run(cache):
        f = ssm.ssm_gated_scan_fwd_ckpt(**t)
        b = ssm.ssm_gated_scan_bwd_ckpt(dy=dy, checkpoints=f[2], **t)
        p = ssm.ssm_gated_scan_packed_fwd(**rows, cu_seqlens=cu, cache=cache)
        s = ssm.ssm_gated_update_cache(cache, None, **one)
        return [*f, *(v for v in b.values() if v is not None), p, s]

    c0 = start.clone()
    eager = run(c0)
    torch.cuda.synchronize()
    c1 = start.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        outs = run(c1)
    torch.cuda.synchronize()
    other = make((2, 900, 40), F, 3)
    for rep in range(4):
        for o in outs:
            o.fill_(3.0)
        c1.copy_(start)
        graph.replay()
        ssm.ssm_gated_scan_fwd(**other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)) and torch.equal(c1, c0), f"replay {rep}"


def test_streams_and_a_given_workspace():
    """Two calls at once on two streams, each with its workspace; the results are the eager ones."""
    a, b = make((2, 1500, 128), BF, 31), make((2, 1500, 128), BF, 32)
    ya, yb = ssm.ssm_gated_scan_fwd(**a)[0], ssm.ssm_gated_scan_fwd(**b)[0]
    n = ssm.ssm_gated_scan_workspace(2, 1500, 128, BF)
    assert n > 0
    w = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        outs.append((ssm.ssm_gated_scan_fwd(**a, workspace=w[0], stream=s[0])[0],
                     ssm.ssm_gated_scan_fwd(**b, workspace=w[1], stream=s[1])[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(p, ya) and torch.equal(q, yb) for p, q in outs)
    with pytest.raises(ssm.SsmError, match="workspace"):
        ssm.ssm_gated_scan_fwd(**a, workspace=w[0][:n - 16])


def test_empty_calls():
    t = make((2, 0, 12), F, 1)
    h0 = torch.randn(2, 12).cuda()
    y, last, saved = ssm.ssm_gated_scan_fwd_ckpt(**t, initial_state=h0)
    assert y.shape == (2, 0, 12) and torch.equal(last, h0) and saved.shape == (0, 12)
    assert (ssm.ssm_gated_scan_fwd(**t)[1] == 0).all()
    grads = ssm.ssm_gated_scan_bwd_ckpt(**t, dy=t["x"], checkpoints=saved, initial_state=h0, dlast_state=h0 * 2)
    assert torch.equal(grads["dinitial_state"], h0 * 2)
    assert all((grads[k] == 0).all() for k in ("da_param", "da_bias", "dx_bias"))
    cache = torch.ones(3, 12).cuda()
    none = {k: (v[0] if v is not None and v.dim() == 3 else v) for k, v in t.items()}
    ssm.ssm_gated_scan_packed_fwd(**none, cu_seqlens=torch.zeros(3, dtype=torch.int32).cuda(), cache=cache)
    ssm.ssm_gated_update_cache(cache, None, **none)
    assert (cache == 1).all()


def test_offsets_past_32_bits():
    """The last of many rows of a wide tensor: over 2^31 elements, over 2^32 bytes."""
    dim, total = 32768, 66000
    assert total * dim > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(total, dim, generator=g, device="cuda", dtype=BF)
    param = torch.full((dim,), -5.0).cuda()
    cut = total - 150
    cu = torch.tensor([0, cut, total], dtype=torch.int32).cuda()
    y = ssm.ssm_gated_scan_packed_fwd(x, x, x, param, cu)
    alone = ssm.ssm_gated_scan_packed_fwd(*(x[cut:].contiguous(),) * 3, param, torch.tensor([0, 150], dtype=torch.int32).cuda())
    d = x[cut:, -8:].cpu().double()
    yr, ey, _, _ = R.forward(d, d, d, param[-8:].cpu().double())
    R.check(y[cut:, -8:], yr, ey, BF, "last rows")
    R.check(alone[:, -8:], yr, ey, BF, "the same rows alone")
