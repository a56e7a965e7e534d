"""GPU: the paged-cache operators where scores jump, are infinite, or where a
call's surroundings (streams, captures, many blocks in a row) could show.

Tolerances are those of test_gpu_paged.py; where the scores are exact dot
products (one dimension only) a score's error is that of its scaling,
4 u32 |s|.
"""
import math

import pytest
import torch

from tests.test_gpu_paged import DT, U32, Batch, code, pe  # noqa: F401

pytestmark = pytest.mark.gpu


def compare(b, out, lse, i, d=None, rows=None):
    """Request i's rows against the 64-bit form; d: the scores' error bound
    (None: that of a dot product of hd terms, over the finite keys)."""
    s = torch.cat([b.slots_prefix(), b.slots(i)])
    G, n, r0 = b.nq // b.nkv, b.n[i], b.off_h[i]
    kk = b.k.view(-1, b.nkv, b.hd)[s].double().repeat_interleave(G, 1)
    vv = b.v.view(-1, b.nkv, b.hd)[s].double().repeat_interleave(G, 1)
    qq = b.q[r0:r0 + n].double()
    seen = torch.arange(len(s), device="cuda") <= b.P + b.c[i] + torch.arange(n, device="cuda")[:, None]
    dots = torch.where(seen, torch.einsum("rhd,khd->hrk", qq, kk) * b.scale, -math.inf)
    top = dots.amax(-1, keepdim=True)
    p = torch.exp(dots - top)
    z = p.sum(-1, keepdim=True)
    p = p / z
    ref, A = torch.einsum("hrk,khd->rhd", p, vv), torch.einsum("hrk,khd->rhd", p, vv.abs())
    rl = (top + torch.log(z))[..., 0].T
    if d is None:
        finite = torch.where(kk.isfinite(), kk.abs(), 0.0)
        mag = torch.where(seen, torch.einsum("rhd,khd->hrk", qq.abs(), finite), 0.0).amax(-1) * b.scale
        d = ((b.hd + 2) * U32 * mag).T
    u, keys = torch.finfo(b.dt).eps / 2, len(s)
    w = (2 * d + 2.0 ** -21 + 2 * keys * U32)
    w = w[..., None] if torch.is_tensor(w) else w
    tol = (w + (u if b.dtype == "bf16" else 0.0)) * A + u * (ref.abs() + A * w) + 1e-30
    got = out[r0:r0 + n].double()
    sel = slice(None) if rows is None else rows
    ratio = ((got - ref).abs() / tol)[sel]
    assert not ratio.isnan().any() and (ratio <= 1).all(), (i, float(ratio.nan_to_num(1e9).max()))
    if lse is not None:
        err = (lse[r0:r0 + n].double() - rl).abs() / (d + 2 * keys * U32 + 2.0 ** -21 + 4 * U32 * rl.abs())
        assert (err[sel] <= 1).all(), (i, float(err[sel].max()))


# ---------------------------------------------------------- running maximum
def tiles_in_a_row(b):
    """The bf16 kernel's line of key tiles, cut among its CTAs: how many tiles
    of one unit a CTA takes, at the median over the CTAs (the kernel's costs:
    19 a tile against one query tile, 31 against two; units 50 and 100)."""
    G = b.nq // b.nkv
    RT, pt, T = 128 // G, -(-b.P // 128), b.T
    packed = -(-T // RT)
    apart = b.B * -(-(-(-T // b.B)) // RT)
    shared = b.P > 0 and (apart - packed) * pt > 4 * packed
    units = []
    if shared:
        units += [(pt, min(2 * RT, T - r) > RT) for _ in range(b.nkv) for r in range(0, T, 2 * RT)]
    for n, c in zip(b.n, b.c):
        units += [((0 if shared else pt) + -(-(c + min(n, r + 2 * RT)) // 128), min(2 * RT, n - r) > RT)
                  for _ in range(b.nkv) for r in range(0, n, 2 * RT)]
    total = sum((100 if two else 50) + t * (31 if two else 19) for t, two in units)
    part = total / torch.cuda.get_device_properties(0).multi_processor_count
    best, x = {}, 0
    for t, two in units:
        own, w = (100, 31) if two else (50, 19)
        count = {}
        for i in range(t):
            c = int((x + (own + i * w if i else 0)) / part)
            count[c] = count.get(c, 0) + 1
        for c, k in count.items():
            best[c] = max(best.get(c, 0), k)
        x += own + t * w
    run = sorted(best.values())
    return run[len(run) // 2], {two for _, two in units}


JUMPS = [
    # nq, nkv, hd, page, prefix, rows, cached; tiles a CTA takes of a unit; units of two query tiles among them
    ((8, 8, 64, 16, 0, [1], [20000]), 6, False),
    ((32, 8, 128, 64, 0, [4], [20000]), 6, False),
    ((32, 8, 128, 16, 0, [64], [20000]), 6, True),
    ((16, 8, 64, 64, 0, [200], [15000]), 6, True),
    ((32, 8, 128, 16, 20000, [2] * 8, [5 * i for i in range(8)]), 6, False),   # packed against the prefix
    ((32, 8, 64, 32, 20000, [1] * 64, [3 * i for i in range(64)]), 6, True),
    ((8, 2, 128, 16, 300, [8] * 40, [2000 + 31 * i for i in range(40)]), 6, False),
]


@pytest.mark.parametrize("jump", [50, 100, 300])
@pytest.mark.parametrize("case,need,two", JUMPS, ids=lambda c: str(c[:5]) if isinstance(c, tuple) else None)
def test_maxima_that_jump_between_tiles(pe, case, need, two, jump):
    """Scores rise by `jump` nats from a key tile to the next (16 levels, then
    from the bottom again; the odd heads fall): what was summed under the old
    maximum must vanish, however far below it lies."""
    b = Batch("bf16", *case, seed=20)
    run, kinds = tiles_in_a_row(b)
    assert run >= need and two in kinds, (run, kinds)   # a stream meets several tiles of a unit
    b.scale = 0.125
    sign = 1.0 - 2.0 * (torch.arange(b.nq, device="cuda") % 2)
    b.q.zero_()
    b.q[:, :, 0] = 8.0 * jump * sign
    kf, vf = b.k.view(-1, b.nkv, b.hd), b.v.view(-1, b.nkv, b.hd)
    for s in [b.slots_prefix()] + [b.slots(i) for i in range(b.B)]:
        tile = torch.arange(len(s), device="cuda") // 128
        kf[s] = 0.0
        kf[s, :, 0] = (tile % 16).to(b.dt)[:, None]
        vf[s] += (1 + tile % 3).to(b.dt)[:, None, None]
    pe.peagle_clear_library_status()
    out, lse = b.attend(pe)
    assert pe.peagle_get_library_status() == 0
    for i in range(b.B):
        compare(b, out, lse, i, d=4 * U32 * 15 * jump)


@pytest.mark.parametrize("case", [(8, 2, 128, 16, 0, [3] * 64, [4000 + 9 * i for i in range(64)]),
                                  (8, 2, 64, 64, 0, [150] * 4, [9000, 7000, 8000, 6000]),
                                  (8, 2, 128, 32, 12000, [5] * 30, [40 * i for i in range(30)])],
                         ids=lambda c: str(c[:5]))
def test_sharp_scores_over_many_tiles(pe, case):
    b = Batch("bf16", *case, qgain=30.0, seed=21)
    assert tiles_in_a_row(b)[0] >= 4
    out, lse = b.attend(pe)
    for i in range(b.B):
        compare(b, out, lse, i)


# ------------------------------------------------- hidden and infinite values
@pytest.mark.parametrize("rows,cached", [([2, 5, 3, 9] * 500, [7, 130, 0, 300] * 500),    # units of one query tile
                                         ([40, 70, 64, 33] * 40, [7, 130, 200, 300] * 40)])   # and of two
def test_hidden_values_in_many_units_in_a_row(pe, rows, cached):
    """Every request's last token holds a NaN value: the mark that a unit has
    met one may not be lost to the next unit's."""
    b = Batch("bf16", 16, 4, 64, 16, 0, rows, cached, seed=22)
    want, _ = b.attend(pe)
    last = torch.stack([b.slots(i)[-1] for i in range(b.B)])
    b.v.view(-1, 4, 64)[last] = float("nan")
    ends = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    ends[b.off[1:].long() - 1] = True
    first = None
    for _ in range(10):
        out, _ = b.attend(pe)
        assert out[ends].isnan().all() and not out[~ends].isnan().any()
        first = out if first is None else first
        assert torch.equal(out[~ends], first[~ends])
    # the same rows without the NaN, each sum in another order: both within u16 A + roundings, A <= max|v|
    A = float(b.v.nan_to_num(0).abs().max())
    assert ((first[~ends].float() - want[~ends].float()).abs() <= 4 * 2.0 ** -8 * A).all()


@pytest.mark.parametrize("hidden", [False, True])
@pytest.mark.parametrize("lead", [1, 130])
@pytest.mark.parametrize("case", [("bf16", 8, 2, 128, 16, 0, [4, 2], [200, 3000]),
                                  ("bf16", 8, 2, 64, 32, 200, [5, 40], [3, 150]),
                                  ("f32", 8, 2, 128, 16, 0, [4, 2], [200, 3000]),
                                  ("f32", 10, 2, 64, 32, 200, [5, 40], [3, 150]),
                                  ("f32", 96, 1, 64, 16, 0, [4, 2], [200, 190]),
                                  ("f32", 96, 1, 64, 16, 140, [4, 2], [20, 190])],
                         ids=lambda c: f"{c[0]}-q{c[1]}kv{c[2]}hd{c[3]}-x{c[5]}")
def test_leading_keys_whose_score_is_minus_infinity(pe, case, lead, hidden):
    """Their weight is 0 on every path, and where a hidden NaN value is met."""
    b = Batch(*case, seed=23)
    b.q[:, :, 0] = b.q[:, :, 0].abs() + 0.5
    kf = b.k.view(-1, b.nkv, b.hd)
    for i in range(b.B):
        s = torch.cat([b.slots_prefix(), b.slots(i)])[:lead]
        kf[s] = 0.0
        kf[s, :, 0] = -math.inf
    if hidden:
        for i in range(b.B):
            b.v.view(-1, b.nkv, b.hd)[b.slots(i)[-1]] = float("nan")
    out, lse = b.attend(pe)
    if hidden:
        b.n = [x - 1 for x in b.n]   # the rows before the last
    for i in range(b.B):
        compare(b, out, lse, i)


@pytest.mark.parametrize("case", [("bf16", 8, 2, 128, 16, 40, [4, 70], [200, 10]), ("f32", 8, 2, 64, 16, 40, [4, 70], [200, 10]),
                                  ("f32", 96, 1, 64, 16, 40, [4, 2], [200, 10])], ids=lambda c: f"{c[0]}-q{c[1]}")
def test_smallest_scale(pe, case):
    """The smallest scale that is taken makes every score 0 but for 2^-100:
    a plain average of what a row sees."""
    b = Batch(*case, seed=29)
    b.scale = 2.0 ** -126
    out, lse = b.attend(pe)
    for i in range(b.B):
        compare(b, out, lse, i, d=2.0 ** -100)


def test_lse_does_not_depend_on_who_finished_the_row(pe):
    """All scores 0: the sum is the number of keys, exactly, and lse its
    logarithm, the same bits from a row that one CTA finishes and from one
    that is joined from a prefix's piece and its own."""
    keys = list(range(2, 300))
    alone = Batch("bf16", 4, 1, 64, 16, 0, [1] * len(keys), [k - 1 for k in keys], qgain=0.0, seed=24)
    joined = Batch("bf16", 4, 1, 64, 16, 1, [1] * len(keys), [k - 2 for k in keys], qgain=0.0, seed=24)
    _, a = alone.attend(pe)
    _, j = joined.attend(pe)
    want = torch.log(torch.tensor(keys, dtype=torch.float64, device="cuda"))[:, None]
    for x in (a, j):   # a logarithm off by a unit in the last place (2 u32), a rounded constant and product
        assert ((x.double() - want).abs() <= 4 * U32 * want).all()
    assert torch.equal(a, j)


# ------------------------------------------------------------ surroundings
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_operators_on_a_side_stream(pe, dtype):
    """Append and attention on another stream behind work that is still on its
    way there: buffers are filled on that stream, and nothing runs elsewhere."""
    b = Batch(dtype, 8, 2, 128, 16, 200, [3, 150], [40, 300], seed=25)
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(b.T, 12 * 128, generator=g, device="cuda")
    pos = torch.arange(b.T, device="cuda", dtype=torch.int32)
    cos, sin = (torch.empty(b.T, 64, device="cuda") for _ in range(2))
    pe.peagle_rope_table(b.T, 128, 1e4, cos, sin)

    def chain(stream):
        q = torch.full((b.T, 8, 128), 7.0, device="cuda").to(b.dt)
        pe.peagle_kv_append(code(pe, dtype), 0, b.T, b.B, 8, 2, 128, x, b.off, pos, cos, sin, b.T, b.ps, b.num_pages,
                            b.max_pages, b.table, b.kv, q, b.k, b.v, stream)
        b.q = q
        return b.attend(pe, stream=stream)

    x = qkv
    want, wl = chain(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = torch.zeros_like(qkv)
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(4):
            big = big @ big / 64   # keeps the stream busy
        x.copy_(qkv)
        got, gl = chain(s)
    s.synchronize()
    assert torch.equal(want, got) and torch.equal(wl, gl)


def paged_setup(wl, B, prefix, own, seed):
    """Pages of a step's caches: random K/V of the prefix and every request's
    own tokens, in shuffled pages; also the same tokens as one list each."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nkv, hd, ps, dt = wl.num_kv_heads, wl.head_dim, 16, DT[wl.dtype]
    per = 12
    total = B * per * 2 + 8
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    kp, vp = (torch.randn(total, ps, nkv, hd, generator=g, device="cuda").to(dt) for _ in range(2))
    npre = -(-prefix // ps)
    pre, table = perm[:npre].contiguous(), perm[npre:npre + B * per].view(B, per).contiguous()
    full = perm[npre + B * per:npre + 2 * B * per].view(B, per).contiguous()
    for t in (kp, vp):
        f = t.view(-1, nkv, hd)
        for b in range(B):
            src = [pre[i // ps].long() * ps + i % ps for i in range(prefix)]
            src += [table[b, i // ps].long() * ps + i % ps for i in range(own[b])]
            dst = [full[b, i // ps].long() * ps + i % ps for i in range(prefix + own[b])]
            f[torch.stack(dst)] = f[torch.stack(src)]
    return kp, vp, pre, table, full


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_loop_behind_a_prefix(pe, dtype):
    """Three rounds of the loop behind a shared prefix against the loop whose
    requests hold the prefix's tokens as their own. Rotary positions count the
    prefix, kv_lens do not."""
    import synth
    from eagle_speculative_drafting_gb300.loop import PagedDraftLoop
    from tests import harness
    B, P, own = 3, 45, [40, 17, 64]
    wl = synth.WORKLOADS["tiny_f32_decode"].scaled(dtype=dtype, batch=B)
    model = harness.make_model(wl, synth.make_weights(wl))
    kp, vp, pre, table, full = paged_setup(wl, B, P, own, 26)
    lens = torch.tensor(own, dtype=torch.int32, device="cuda")
    a = PagedDraftLoop(model, wl.K, [kp.clone()], [vp.clone()], full, lens + P)
    p = PagedDraftLoop(model, wl.K, [kp], [vp], table, lens, pre, P)
    for loop in (a, p):
        loop.start([1, 2, 3], [P + x for x in own])
    g = torch.Generator(device="cuda").manual_seed(2)
    for rnd in range(3):
        aux = torch.randn(a.total_new, wl.num_aux * wl.target_hidden, generator=g, device="cuda").to(DT[dtype])
        la, lp = (torch.empty(B, wl.K, wl.vocab, device="cuda") for _ in range(2))
        a.draft(aux, la)
        p.draft(aux, lp)
        assert harness.max_abs_rel(lp.cpu().numpy(), la.cpu().numpy()) <= (1e-4 if dtype == "f32" else 2e-2)
        p.drafts.copy_(a.drafts)   # (near ties may fall either way in bf16)
        tgt = torch.zeros(B, wl.K + 1, dtype=torch.int32, device="cuda")
        tgt[:, :wl.K] = a.drafts
        for b in range(B):
            keep = (b + rnd) % (wl.K + 1)
            if keep < wl.K:
                tgt[b, keep] = (a.drafts[b, keep] + 1) % wl.vocab
        for loop in (a, p):
            loop.verify_greedy(tgt)
        assert torch.equal(a.kv_lens, p.kv_lens + P) and torch.equal(a.new_pos, p.new_pos)
    assert pe.peagle_get_device_status(model.handle) == 0
    model.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_paged_step(pe, dtype):
    """A captured paged step replays beside eager steps of other sizes, which
    take other workspaces, and follows the lengths that the device holds."""
    import synth
    from tests import harness
    B, P, own = 3, 45, [40, 17, 64]
    wl = synth.WORKLOADS["tiny_f32_decode"].scaled(dtype=dtype, batch=B)
    model = harness.make_model(wl, synth.make_weights(wl))
    kp, vp, pre, table, _ = paged_setup(wl, B, P, own, 27)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(3)
    aux = torch.randn(6, wl.num_aux * wl.target_hidden, generator=g, device="cuda").to(DT[dtype])
    off, tok, pos, kv = i32([0, 1, 4, 6]), i32([3, 1, 4, 1, 5, 9]), i32([85, 62, 63, 64, 109, 110]), i32(own)
    logits = torch.empty(B, wl.K, wl.vocab, device="cuda")

    def step(logits):
        return model.draft_step_paged(wl.K, off, aux, tok, pos, [kp], [vp], table, kv, pre, P, logits=logits)

    def eager():
        x = torch.empty_like(logits)
        t = step(x)
        return x, t

    want, wt = eager()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        toks = step(logits)
    for lens in (own, [30, 10, 50]):
        kv.copy_(i32(lens))
        pos.copy_(i32([lens[0] + P] + [lens[1] + P + j for j in range(3)] + [lens[2] + P + j for j in range(2)]))
        want, wt = eager()
        # a larger step between, over the same pages' scratch
        n = 300
        model.draft_step_paged(wl.K, i32([0, n]), aux[:1].expand(n, -1).contiguous(), tok[:1].expand(n).contiguous(),
                               torch.arange(n, device="cuda", dtype=torch.int32), [kp.clone()], [vp.clone()],
                               torch.arange(40, device="cuda", dtype=torch.int32)[None].contiguous(), i32([0]))
        logits.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(logits, want) and torch.equal(toks, wt)
    assert pe.peagle_get_device_status(model.handle) == 0
    model.close()


def test_paged_step_workspace_holds_what_the_step_uses(pe):
    """fp32, per row: layer inputs, activations, q, the attention's output, the
    residual stream, one contraction's output; and the attention's workspace."""
    import synth
    from tests import harness
    wl = synth.WORKLOADS["tiny_f32_decode"]
    model = harness.make_model(wl, synth.make_weights(wl))
    c, B, K = model.cfg, 2, 4
    qh, kvh = c.num_q_heads * c.head_dim, c.num_kv_heads * c.head_dim
    for N in (2, 500, 8000):
        rows = N + B * (K - 1)
        part = max(N * c.hidden, rows * (qh + 2 * kvh), rows * c.hidden, rows * 2 * c.intermediate,
                   B * K * c.draft_vocab)
        floats = N * 3 * c.hidden + rows * (2 * c.hidden + c.intermediate + 2 * qh) + part
        most = 4 * floats + pe.peagle_paged_attention_workspace_size(0, rows, B, c.num_q_heads, c.num_kv_heads,
                                                                     c.head_dim, 100)
        most += 8 * B * K * (c.draft_vocab // 8 + 64) + 20 * 256   # argmax partials; roundings to 256 bytes
        assert pe.peagle_draft_step_paged_workspace_size(model.handle, B, K, N, 100) <= most
    model.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 4])
def test_step_flags_a_request_without_rows(pe, dtype, K):
    """Every request of a step brings a row: one without is flagged, and the
    others' drafts are as if it were not there."""
    import synth
    from tests import harness
    wl = synth.WORKLOADS["tiny_f32_decode"].scaled(dtype=dtype, batch=3)
    model = harness.make_model(wl, synth.make_weights(wl))
    own = [40, 17, 64]
    kp, vp, pre, table, _ = paged_setup(wl, 3, 45, own, 28)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    aux = torch.randn(4, wl.num_aux * wl.target_hidden, device="cuda").to(DT[dtype])

    def step(off):
        logits = torch.zeros(3, K, wl.vocab, device="cuda")
        model.draft_step_paged(K, i32(off), aux, i32([3, 1, 4, 1]), i32([85, 86, 109, 110]), [kp.clone()], [vp.clone()],
                               table, i32(own), pre, 45, logits=logits)
        torch.cuda.synchronize()
        status = pe.peagle_get_device_status(model.handle)
        pe.peagle_clear_device_status(model.handle)
        return logits, status

    _, status = step([0, 2, 3, 4])
    assert status == 0
    bad, status = step([0, 2, 2, 4])
    assert status == pe.PEAGLE_DEV_BOUNDS
    assert bad[0].isfinite().all() and bad[2].isfinite().all()
    model.close()


@pytest.mark.parametrize("dtype,nq", [("bf16", 8), ("f32", 8), ("f32", 96)])
def test_attention_flags_a_malformed_request_without_rows(pe, dtype, nq):
    """Its lengths are wrong and it has no row: flagged on every path, and the
    other requests' rows are right."""
    b = Batch(dtype, nq, 1, 64, 16, 20, [3, 0, 2], [40, 5, 30], seed=30)
    b.kv[1] = -1
    pe.peagle_clear_library_status()
    out, lse = b.attend(pe)
    assert pe.peagle_get_library_status() == pe.PEAGLE_DEV_BOUNDS
    pe.peagle_clear_library_status()
    for i in (0, 2):
        compare(b, out, lse, i)


HIDDEN = [("bf16", 8, 2, 128, 16, 0, [5, 3], [200, 10]),            # one query tile, joined streams
          ("bf16", 8, 2, 64, 32, 0, [9, 1, 30], [5000, 4000, 7000]),   # pieces of several CTAs
          ("bf16", 32, 8, 128, 16, 300, [64, 150, 7], [20, 100, 600]),   # two query tiles behind a prefix
          ("bf16", 8, 8, 64, 16, 0, [256, 130], [60, 3]),           # 256 rows to a unit
          ("bf16", 8, 2, 128, 16, 9000, [4] * 30, [3 * i for i in range(30)]),   # packed against the prefix
          ("bf16", 128, 1, 64, 16, 10, [3, 2], [130, 5]),
          ("f32", 8, 2, 128, 16, 0, [5, 3], [200, 10]),
          ("f32", 10, 2, 64, 32, 130, [70, 9, 30], [900, 40, 700])]


@pytest.mark.parametrize("case", HIDDEN, ids=lambda c: f"{c[0]}-q{c[1]}kv{c[2]}hd{c[3]}-x{c[5]}")
def test_hidden_elements_touch_only_their_rows_and_columns(pe, case):
    """Infinite and NaN elements of tokens that the first rows do not see: in
    the rows that see them their columns are what a sum with them is, and every
    other bit of the result is as if they were finite."""
    b = Batch(*case, seed=31)
    vf = b.v.view(-1, b.nkv, b.hd)
    want, wl = b.attend(pe)
    expect = want.clone()
    G = b.nq // b.nkv
    for i in range(b.B):
        n, r0 = b.n[i], b.off_h[i]
        if n < 2:
            continue
        s = b.slots(i)[b.c[i]:]
        first, last = n // 2, n - 1   # rows whose tokens get odd elements (one row when n == 2)
        for row, col, value in ((first, 3, math.inf), (last, 3, math.inf), (first, 17, -math.inf), (last, 30, math.nan),
                                (last, 17, math.inf if last > first else -math.inf)):
            vf[s[row], 0, col] = value
        heads = slice(0, G)   # of key head 0
        expect[r0 + first:r0 + n, heads, 3] = math.inf
        expect[r0 + first:r0 + n, heads, 17] = -math.inf
        expect[r0 + last, heads, 30] = math.nan
        if last > first:
            expect[r0 + last, heads, 17] = math.nan
    out, lse = b.attend(pe)
    kind = torch.int16 if b.dtype == "bf16" else torch.int32
    nan = expect.isnan()
    assert torch.equal(out.isnan(), nan)
    assert torch.equal(out[~nan].view(kind), expect[~nan].view(kind)) and torch.equal(lse, wl)


def test_hidden_values_do_not_hold_up_the_batch(pe):
    """One request's bad value behind a long prefix: the call takes about as
    long as without it (computing the block's rows again, one key at a time,
    took hundreds of times as long)."""
    b = Batch("bf16", 32, 8, 128, 64, 20000, [8] * 40, [10 * i for i in range(40)], seed=32)

    def time(reps=5):
        best = 1e9
        for _ in range(reps):
            x, y = torch.cuda.Event(True), torch.cuda.Event(True)
            x.record()
            b.attend(pe)
            y.record()
            torch.cuda.synchronize()
            best = min(best, x.elapsed_time(y))
        return best
    time()
    plain = time()
    b.v.view(-1, 8, 128)[b.slots(7)[-1]] = float("nan")
    assert time() <= 5 * plain + 1.0   # ms
