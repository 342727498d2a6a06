"""Attention over packed sequences, its gradients, chunks over the paged cache and rotary positions with
several axes on the GPU, against the plain fp64 forms of packed_ref.py within their derived bounds."""
import random
import types

import pytest
import torch

import packed_ref
from exact_attention_161_b200 import synth

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _batch(lens, Hq, Hkv, D, seed, before=0, after=0, fused=False):
    """q, k, v, dout, offsets (list and device tensor); `before` and `after` rows outside every sequence hold
    NaN. fused: q, k, v are views of one tensor."""
    g = _gen(seed)
    T = before + sum(lens) + after
    starts = [before]
    for n in lens:
        starts.append(starts[-1] + n)
    if fused:
        x = _randn(g, T, Hq + 2 * Hkv, D)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        q, k, v = _randn(g, T, Hq, D), _randn(g, T, Hkv, D), _randn(g, T, Hkv, D)
    dout = _randn(g, T, Hq, D)
    for x in (q, k, v, dout):
        x[:before] = NAN
        x[T - after:] = NAN
    return q, k, v, dout, starts, torch.tensor(starts, dtype=torch.int32, device="cuda")


def _check_batch(api, lens, Hq, Hkv, D, causal, window, seed, scale=0.0, train=True, **kw):
    q, k, v, dout, starts, cu = _batch(lens, Hq, Hkv, D, seed, **kw)
    T = q.shape[0]
    o = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, T), 7.0, device="cuda")
    api.attn_packed_fwd(q, k, v, cu, causal=causal, window=window, scale=scale, o=o, lse=lse)
    torch.cuda.synchronize()
    assert api.device_status() == 0
    ref = packed_ref.packed(q, k, v, starts, causal, window, scale or None, dout if train else None)
    packed_ref.check("o", o, ref)
    packed_ref.check("lse", lse, ref)
    outside = torch.ones(T, dtype=torch.bool, device="cuda")
    outside[starts[0]:starts[-1]] = False
    assert bool((o[outside] == 7).all()) and bool((lse[:, outside] == 7).all())
    if not train:
        return
    grads = [torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (q, k, v)]
    api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=causal, window=window, scale=scale, dq=grads[0], dk=grads[1],
                        dv=grads[2])
    torch.cuda.synchronize()
    assert api.device_status() == 0
    for name, x in zip(("dq", "dk", "dv"), grads):
        packed_ref.check(name, x, ref)
        assert bool((x[outside] == 7).all()), name


# lengths around every border: one token, 16-row slices, TT-token tiles, 128-key tiles, 64- and 256-token blocks
LENS = [1, 0, 15, 16, 17, 63, 64, 65, 0, 127, 128, 129, 255, 256, 257, 2, 400]


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64), (12, 4, 64), (8, 1, 128), (10, 2, 64), (4, 4, 128),
                                      (14, 2, 128), (32, 1, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100)])
def test_packed_lengths_and_heads(cuda_api, Hq, Hkv, D, causal, window):
    _check_batch(cuda_api, LENS, Hq, Hkv, D, causal, window, seed=Hq * 7 + Hkv + D)


@pytest.mark.parametrize("window", [1, 2, 16, 127, 128, 129, 500, 2147483647])
def test_packed_windows(cuda_api, window):
    _check_batch(cuda_api, [300, 1, 129, 700], 6, 2, 64, True, window, seed=window % 1000)


@pytest.mark.parametrize("n", [1, 2, 7, 16, 127, 128, 129, 513])
def test_packed_single_sequence(cuda_api, n):
    _check_batch(cuda_api, [n], 8, 2, 128, True, 0, seed=n)
    _check_batch(cuda_api, [n], 3, 3, 64, False, 0, seed=n + 1)


def test_packed_views_and_rows_of_nobody(cuda_api):
    """q, k, v as views of one projection; NaN rows in front of the first and behind the last sequence."""
    for D, (Hq, Hkv) in ((128, (8, 2)), (64, (6, 2)), (64, (4, 4))):
        for causal in (True, False):
            _check_batch(cuda_api, [33, 0, 140, 77, 1], Hq, Hkv, D, causal, 0, seed=D + Hq, before=5, after=11,
                         fused=True)


def test_packed_neighbours_of_nan_sequences(cuda_api):
    """A sequence full of NaN spoils its own rows only."""
    lens = [40, 37, 90]
    q, k, v, dout, starts, cu = _batch(lens, 8, 2, 128, 3)
    for x in (q, k, v, dout):
        x[40:77] = NAN
    o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True)
    grads = cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True)
    for a, b in ((0, 40), (77, 167)):
        ref = packed_ref.attend(q[a:b], k[a:b], v[a:b], True, 0, dout=dout[a:b])
        packed_ref.check("o", o[a:b], ref)
        packed_ref.check("lse", lse[:, a:b], ref)
        for name, x in zip(("dq", "dk", "dv"), grads):
            packed_ref.check(name, x[a:b], ref)
    assert bool(torch.isnan(o[40:77].float()).all())


@pytest.mark.parametrize("D", [64, 128])
def test_packed_many_heads_per_group(cuda_api, D):
    """One token per tile (128 query heads on one K/V head), and a group that does not divide 128."""
    _check_batch(cuda_api, [3, 130, 20], 128, 1, D, True, 0, seed=D)
    _check_batch(cuda_api, [3, 130, 20], 100, 1, D, True, 30, seed=D + 1, train=False)


def test_packed_scale_and_no_lse(cuda_api):
    _check_batch(cuda_api, [50, 200], 4, 2, 64, True, 0, seed=9, scale=0.02)
    q, k, v, _, _, cu = _batch([50, 200], 4, 2, 64, 9)
    a, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True, scale=0.02)
    b, none = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True, scale=0.02, want_lse=False)
    assert none is None and torch.equal(a, b)


def test_packed_cut_keys_repeat_bit_for_bit(cuda_api):
    """Few long sequences: the keys of a block are cut into parts; repeats give the same bits."""
    q, k, v, dout, starts, cu = _batch([2500, 1, 3000], 2, 1, 128, 11)
    for causal, window in ((True, 0), (False, 0), (True, 1700)):
        o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=causal, window=window)
        ref = packed_ref.packed(q, k, v, starts, causal, window)
        packed_ref.check("o", o, ref)
        packed_ref.check("lse", lse, ref)
        g0 = cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=causal, window=window)
        for _ in range(3):
            o2, lse2 = cuda_api.attn_packed_fwd(q, k, v, cu, causal=causal, window=window)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
            g = cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=causal, window=window)
            assert torch.equal(g0[1], g[1]) and torch.equal(g0[2], g[2])
    assert cuda_api.device_status() == 0


def test_packed_many_sequences(cuda_api):
    """More sequences than the plan keeps in shared memory, most of them tiny."""
    rng = random.Random(4)
    lens = [rng.choice([0, 1, 1, 2, 3, 9]) for _ in range(2500)]
    _check_batch(cuda_api, lens, 4, 2, 64, True, 0, seed=12)


def test_packed_equals_the_batched_forward(cuda_api):
    """Equal lengths: the same attention as attn_fwd and attn_bwd, within both calls' bounds."""
    B, Hq, Hkv, N, D = 2, 8, 2, 384, 128
    q, k, v = (x.cuda() for x in synth.prefill_inputs(B, Hq, Hkv, N, D, seed=31))
    dout = _randn(_gen(32), B, Hq, N, D)
    o, lse = cuda_api.attn_fwd(q, k, v, causal=True)
    grads = cuda_api.attn_bwd(q, k, v, o, lse, dout, causal=True)
    flat = lambda x: x.transpose(1, 2).reshape(B * N, x.shape[1], D)
    cu = torch.tensor([0, N, 2 * N], dtype=torch.int32, device="cuda")
    qp, kp, vp, dp = flat(q), flat(k), flat(v), flat(dout)
    o2, lse2 = cuda_api.attn_packed_fwd(qp, kp, vp, cu, causal=True)
    grads2 = cuda_api.attn_packed_bwd(qp, kp, vp, o2, lse2, dp, cu, causal=True)
    ref = packed_ref.packed(qp, kp, vp, [0, N, 2 * N], True, 0, dout=dp)
    for name, a, b in zip(("o", "dq", "dk", "dv"), (o,) + tuple(grads), (o2,) + tuple(grads2)):
        assert bool(((flat(a).double() - b.double()).abs() <= 2 * ref[name + "_tol"]).all()), name
    assert (lse.transpose(0, 1).reshape(Hq, B * N) - lse2).abs().max() < 2e-3


def test_packed_gradient_against_differences(cuda_api):
    """The kernel's gradients against a difference quotient of the plain forward along a random direction:
    sum(grad * d) is off by at most sum(tol |d|), the quotient by rounding (1e-6)."""
    q, k, v, w, starts, cu = _batch([70, 1, 200], 4, 2, 64, 13)
    o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True)
    grads = cuda_api.attn_packed_bwd(q, k, v, o, lse, w, cu, causal=True)
    ref = packed_ref.packed(q, k, v, starts, True, 0, dout=w)
    xs = [x.double() for x in (q, k, v)]
    for i, name in enumerate(("dq", "dk", "dv")):
        d = torch.randn(xs[i].shape, generator=_gen(14 + i), device="cuda", dtype=torch.float64)
        f = []
        for h in (1e-5, -1e-5):
            y = list(xs)
            y[i] = xs[i] + h * d
            f.append((packed_ref.packed(*y, starts, True, 0)["o"] * w.double()).sum().item())
        got = (grads[i].double() * d).sum().item()
        assert abs((f[0] - f[1]) / 2e-5 - got) <= (ref[name + "_tol"] * d.abs()).sum().item() + 1e-6


def test_bad_offsets_are_reported(cuda_api):
    """Offsets that decrease or leave [0, T] compute nothing and set the status bit."""
    q, k, v, dout, _, _ = _batch([100], 4, 2, 64, 15)
    for bad in ([0, 60, 50, 100], [0, 101], [-1, 50], [0, 2147483647, 100], [0, -2147483648, 100]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o = torch.full((100, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, 100), 7.0, device="cuda")
        cuda_api.attn_packed_fwd(q, k, v, cu, causal=True, o=o, lse=lse)
        assert cuda_api.device_status() == cuda_api.DEVICE_BAD_OFFSETS
        assert bool((o == 7).all()) and bool((lse == 7).all())
        dq, dk, dv = (torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (q, k, v))
        cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True, dq=dq, dk=dk, dv=dv)
        assert cuda_api.device_status() == cuda_api.DEVICE_BAD_OFFSETS
        assert all(bool((x == 7).all()) for x in (dq, dk, dv))
    assert cuda_api.device_status() == 0


# ------------------------------------------------------------------ chunks over the paged cache
def _cache(total, Hkv, D, seed, spare=5, extra_blocks=2):
    """Pages with random values in the slots of each sequence's tokens and NaN in every other slot."""
    g = _gen(seed)
    pages = [(n + 15) // 16 for n in total]
    pool = sum(pages) + spare
    perm = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(total), max(pages) + extra_blocks), -7, dtype=torch.int32)
    kp = torch.full((pool, Hkv, 16, D), NAN, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    at = 0
    for s, n in enumerate(total):
        table[s, :pages[s]] = torch.tensor(perm[at:at + pages[s]], dtype=torch.int32)
        at += pages[s]
        for pg in range(pages[s]):
            m = min(16, n - 16 * pg)
            for x in (kp, vp):
                x[table[s, pg], :, :m] = _randn(g, Hkv, m, D)
    return kp, vp, table


def _rows(x, table, s, n):
    """The first n keys or values of sequence s, [n, Hkv, D]."""
    pages = table[s, :(n + 15) // 16].long().cuda()
    return x[pages].transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n]


def _check_chunk(api, ctx, new, Hq, Hkv, D, window, seed, append=True, scale=0.0, before=0, after=0, fused=False):
    total = [c + n for c, n in zip(ctx, new)]
    kp, vp, table = _cache(total, Hkv, D, seed)
    q, kn, vn, _, starts, cu = _batch(new, Hq, Hkv, D, seed + 1, before=before, after=after, fused=fused)
    T = q.shape[0]
    want_k, want_v = kp.clone(), vp.clone()
    if append:
        for s, (c, n) in enumerate(zip(ctx, new)):
            pos = torch.arange(c, c + n)
            if n:
                pg = table[s][pos // 16].long().cuda()
                want_k[pg, :, (pos % 16).cuda()] = kn[starts[s]:starts[s + 1]]
                want_v[pg, :, (pos % 16).cuda()] = vn[starts[s]:starts[s + 1]]
                kp[pg, :, (pos % 16).cuda()] = NAN
                vp[pg, :, (pos % 16).cuda()] = NAN
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    o = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    api.attn_chunk_paged(q, kp, vp, table.cuda(), lens, cu, k_new=kn if append else None,
                         v_new=vn if append else None, window=window, scale=scale, o=o, lse=lse)
    torch.cuda.synchronize()
    assert api.device_status() == 0
    bits = lambda x: x.view(torch.int16)
    assert torch.equal(bits(kp), bits(want_k)) and torch.equal(bits(vp), bits(want_v))
    worst = 0.0
    for s, n in enumerate(new):
        if n == 0:
            continue
        a, b = starts[s], starts[s + 1]
        ref = packed_ref.attend(q[a:b], _rows(kp, table, s, total[s]), _rows(vp, table, s, total[s]), True, window,
                                scale or None)
        worst = max(worst, packed_ref.check("o", o[a:b], ref), packed_ref.check("lse", lse[a:b].t(), ref))
    outside = torch.ones(T, dtype=torch.bool, device="cuda")
    outside[starts[0]:starts[-1]] = False
    assert bool((o[outside] == 7).all()) and bool((lse[outside] == 7).all())
    return worst


CTX = [0, 1, 15, 16, 100, 127, 128, 500, 1000, 30, 0, 64, 2000]
NEW = [1, 1, 2, 0, 1, 1, 129, 40, 1, 300, 70, 64, 3]


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64), (12, 4, 64), (8, 1, 128), (32, 8, 128), (64, 1, 64)])
@pytest.mark.parametrize("window", [0, 50])
def test_chunk_lengths_and_heads(cuda_api, Hq, Hkv, D, window):
    _check_chunk(cuda_api, CTX, NEW, Hq, Hkv, D, window, seed=Hq + D)


@pytest.mark.parametrize("append", [True, False])
def test_chunk_single_tokens(cuda_api, append):
    """A decode step: one token each, the cache empty, at page borders, and long enough to be cut."""
    ctx = [0, 15, 16, 17, 511, 4000, 127]
    _check_chunk(cuda_api, ctx, [1] * len(ctx), 8, 2, 128, 0, seed=3, append=append)
    _check_chunk(cuda_api, ctx, [1] * len(ctx), 8, 8, 64, 0, seed=4, append=append)
    _check_chunk(cuda_api, [9000], [1], 8, 2, 128, 0, seed=5, append=append)


def test_chunk_long_context(cuda_api):
    _check_chunk(cuda_api, [20000], [70], 4, 1, 128, 0, seed=6)
    _check_chunk(cuda_api, [20000, 50], [3, 500], 4, 2, 64, 5000, seed=7)


def test_chunk_views_scale_and_rows_of_nobody(cuda_api):
    _check_chunk(cuda_api, [100, 7], [30, 90], 4, 2, 128, 0, seed=8, before=3, after=9, fused=True, scale=0.11)


def test_chunk_pages_before_the_window_may_be_gone(cuda_api):
    """Pages wholly before the window of the first new token: entries invalid, memory NaN."""
    for D in (64, 128):
        ctx, n, window = 1000, 20, 200
        kp, vp, table = _cache([ctx + n], 2, D, 9)
        q, kn, vn, _, starts, cu = _batch([n], 8, 2, D, 10)
        pos = torch.arange(ctx, ctx + n)
        pg, slot = table[0][pos // 16].long().cuda(), (pos % 16).cuda()
        kp[pg, :, slot], vp[pg, :, slot] = kn, vn
        ref = packed_ref.attend(q, _rows(kp, table, 0, ctx + n), _rows(vp, table, 0, ctx + n), True, window)
        gone = (ctx - window + 1) // 16
        kp[table[0, :gone].long().cuda()] = NAN
        vp[table[0, :gone].long().cuda()] = NAN
        lens = torch.tensor([ctx + n], dtype=torch.int32, device="cuda")
        for entry in (None, -1, 1 << 30):
            t = table.clone()
            if entry is not None:
                t[0, :gone] = entry
            o, lse = cuda_api.attn_chunk_paged(q, kp, vp, t.cuda(), lens, cu, window=window)
            assert cuda_api.device_status() == 0
            packed_ref.check("o", o, ref)
            packed_ref.check("lse", lse.t(), ref)


def test_chunk_bad_pages_and_lengths_are_reported(cuda_api):
    """A bad table entry: its token is not appended; a bad length: the sequence's rows are NaN. The other
    sequences are as ever. Both are caught by the kernels' own checks before any access."""
    ctx, new = [40, 40, 40, 40], [20, 3, 3, 0]
    total = [c + n for c, n in zip(ctx, new)]
    kp, vp, table = _cache(total, 2, 128, 16)
    q, kn, vn, _, starts, cu = _batch(new, 8, 2, 128, 17)
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    kp0 = kp.clone()
    t = table.clone()
    t[1, 2] = kp.shape[0]
    o, lse = cuda_api.attn_chunk_paged(q, kp, vp, t.cuda(), lens, cu, k_new=kn, v_new=vn)
    assert cuda_api.device_status() == cuda_api.DEVICE_BAD_PAGE
    assert torch.equal(kp[table[1, 2]].view(torch.int16), kp0[table[1, 2]].view(torch.int16))
    good = packed_ref.attend(q[:20], _rows(kp, table, 0, 60), _rows(vp, table, 0, 60), True, 0)
    packed_ref.check("o", o[:20], good)
    for bad in (2, 0, -5, 16 * table.shape[1] + 1, 2147483647):
        kp = kp0.clone()
        lens2 = lens.clone()
        lens2[1], lens2[3] = bad, bad  # sequence 3 brings nothing: its length is not read
        o, lse = cuda_api.attn_chunk_paged(q, kp, vp, table.cuda(), lens2, cu, k_new=kn, v_new=vn)
        assert cuda_api.device_status() == cuda_api.DEVICE_BAD_SEQLEN
        assert bool(torch.isnan(o[20:23].float()).all()) and bool(torch.isnan(lse[20:23]).all())
        assert torch.equal(kp[table[1, 2]].view(torch.int16), kp0[table[1, 2]].view(torch.int16))
        packed_ref.check("o", o[:20], good)
    cu_bad = torch.tensor([0, 20, 18, 26, 26], dtype=torch.int32, device="cuda")
    o = torch.full_like(q, 7.0)
    cuda_api.attn_chunk_paged(q, kp, vp, table.cuda(), lens, cu_bad, o=o)
    assert cuda_api.device_status() == cuda_api.DEVICE_BAD_OFFSETS and bool((o == 7).all())


def test_chunk_equals_the_decode_step(cuda_api):
    """Two new tokens each: the same step as attn_decode_step, and the same pages bit for bit."""
    inp = synth.decode_step_inputs(5, 2, 8, 2, 128, 16, seq_lens=[2, 16, 17, 100, 515], seed=18)
    c = inp.cache
    kp, vp = c.k_pages.cuda(), c.v_pages.cuda()
    o, lse = cuda_api.attn_decode_step(inp.q.cuda(), kp, vp, c.block_table.cuda(), c.seq_lens.cuda(),
                                       k_new=inp.k_new.cuda(), v_new=inp.v_new.cuda())
    kp2, vp2 = c.k_pages.cuda(), c.v_pages.cuda()
    flat = lambda x: x.reshape(-1, *x.shape[2:]).cuda()
    cu = torch.arange(0, 11, 2, dtype=torch.int32, device="cuda")
    o2, lse2 = cuda_api.attn_chunk_paged(flat(inp.q), kp2, vp2, c.block_table.cuda(), c.seq_lens.cuda(), cu,
                                         k_new=flat(inp.k_new), v_new=flat(inp.v_new))
    assert torch.equal(kp.view(torch.int16), kp2.view(torch.int16))
    assert torch.equal(vp.view(torch.int16), vp2.view(torch.int16))
    for s, n in enumerate(c.seq_lens.tolist()):
        ref = packed_ref.attend(flat(inp.q)[2 * s:2 * s + 2], _rows(kp, c.block_table, s, n),
                                _rows(vp, c.block_table, s, n), True, 0)
        packed_ref.check("o", o2[2 * s:2 * s + 2], ref)
        assert bool(((o[s].double() - o2[2 * s:2 * s + 2].double()).abs() <= 2 * ref["o_tol"]).all())


# ------------------------------------------------------------------ rotary positions with several axes
AXES = [([64], False), ([16, 24, 24], False), ([24, 20, 20], True), ([32, 32], False), ([10, 3, 3], True),
        ([1, 2, 3, 2], False), ([16, 16], True), ([32], False)]


@pytest.mark.parametrize("sections,inter", AXES)
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D", [(1, 8, 2, 128), (37, 32, 8, 128), (600, 3, 1, 64), (700, 130, 2, 64)])
def test_rope_axes(cuda_api, sections, inter, half, T, Hq, Hk, D):
    if sum(sections) > D // 2:
        sections = [x // 2 for x in sections]
    g = _gen(T + Hq)
    x = _randn(g, T, Hq + Hk + 1, D)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk]
    for far in (False, True):
        pos = torch.randint(-2 ** 31 if far else 0, 2 ** 31 - 1 if far else 5000, (len(sections), T), generator=g,
                            device="cuda").to(torch.int32)
        for ladder, inverse, ps in ((False, False, 1.0), (True, True, 4.0)):
            a = dict(interleave_axes=inter, per_axis_freq=ladder, rope_half_split=half, rope_base=5e5,
                     rope_pos_scale=ps, inverse=inverse)
            got = cuda_api.attn_rope_axes(q, k, pos, sections, **a)
            for y, src in zip(got, (q, k)):
                want, tol = packed_ref.rope_axes(src, pos, sections, inter, ladder, half, 5e5, ps, inverse)
                tail = 2 * sum(sections)
                assert bool(((y.double() - want).abs() <= tol).all())
                assert torch.equal(y[..., tail:].contiguous().view(torch.int16),
                                   src[..., tail:].contiguous().view(torch.int16))
            only, none = cuda_api.attn_rope_axes(q, None, pos, sections, **a)
            assert none is None and torch.equal(only, got[0])


def test_rope_axes_in_place_keeps_its_neighbours(cuda_api):
    g = _gen(40)
    x = _randn(g, 50, 7, 64)
    before = x.clone()
    pos = torch.arange(50, dtype=torch.int32, device="cuda").repeat(2, 1).contiguous()
    want = cuda_api.attn_rope_axes(x[:, :4], x[:, 4:6], pos, [8, 8], rope_half_split=True)
    q, k = x[:, :4], x[:, 4:6]
    cuda_api.attn_rope_axes(q, k, pos, [8, 8], rope_half_split=True, q_out=q, k_out=k)
    assert torch.equal(x[:, :4], want[0]) and torch.equal(x[:, 4:6], want[1]) and torch.equal(x[:, 6], before[:, 6])


def test_rope_one_axis_is_the_forwards_rotation(cuda_api):
    """One axis and positions 0, 1, ...: packed attention on the rotated rows is attn_fwd with RoPE."""
    N, Hq, Hkv, D = 300, 4, 2, 128
    q, k, v = (x.cuda() for x in synth.prefill_inputs(1, Hq, Hkv, N, D, seed=50))
    o, lse = cuda_api.attn_fwd(q, k, v, causal=True, rope_base=1e4)
    flat = lambda x: x[0].transpose(0, 1).contiguous()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None]
    qr, kr = cuda_api.attn_rope_axes(flat(q), flat(k), pos, [64])
    cu = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    o2, lse2 = cuda_api.attn_packed_fwd(qr, kr, flat(v), cu, causal=True)
    ref = packed_ref.packed(qr, kr, flat(v), [0, N], True, 0)
    packed_ref.check("o", o2, ref)
    # attn_fwd may round a rotated component the other way: its own parity bound on top
    assert bool(((flat(o).double() - o2.double()).abs() <= 2e-2 + ref["o_tol"]).all())
    assert (lse[0] - lse2).abs().max() <= 2e-3


# ------------------------------------------------------------------ together, streams, graphs
def test_a_prompt_in_chunks_then_single_tokens(cuda_api):
    """Rotate, prefill two prompts in ragged chunks over the cache (one of them waits in a step), compare with
    the packed forward of the whole prompts; then attn_decode_paged continues on the same cache."""
    Hq, Hkv, D = 8, 2, 128
    lens = [333, 150]
    q, k, v, _, starts, cu_all = _batch(lens, Hq, Hkv, D, 60)
    T = sum(lens)
    g = torch.Generator().manual_seed(61)
    pos = torch.randint(0, 400, (3, T), generator=g).to(torch.int32).cuda()
    qr, kr = cuda_api.attn_rope_axes(q, k, pos, [16, 24, 24], rope_half_split=True)
    whole, whole_lse = cuda_api.attn_packed_fwd(qr, kr, v, cu_all, causal=True)
    kp, vp, table = _cache([n + 4 for n in lens], Hkv, D, 62)
    kp.fill_(NAN)
    vp.fill_(NAN)
    ref = packed_ref.packed(qr, kr, v, starts, True, 0)
    done, table_d = [0, 0], table.cuda()
    for step in ([100, 1], [0, 64], [17, 85], [216, 0]):
        rows = torch.cat([torch.arange(starts[s] + done[s], starts[s] + done[s] + n) for s, n in enumerate(step)]).cuda()
        cu = torch.tensor([0, step[0], sum(step)], dtype=torch.int32, device="cuda")
        done = [a + b for a, b in zip(done, step)]
        o, lse = cuda_api.attn_chunk_paged(qr[rows], kp, vp, table_d, torch.tensor(done, dtype=torch.int32, device="cuda"),
                                           cu, k_new=kr[rows], v_new=v[rows])
        part = {n: (x[:, rows] if n.startswith("lse") else x[rows]) for n, x in ref.items()}
        packed_ref.check("o", o, part)
        packed_ref.check("lse", lse.t(), part)
        assert bool(((o.double() - whole[rows].double()).abs() <= 2 * part["o_tol"]).all())
    assert done == lens
    q1 = _randn(_gen(63), 2, Hq, D)
    o1, _ = cuda_api.attn_decode_paged(q1, kp, vp, table_d, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for s, n in enumerate(lens):
        one = packed_ref.attend(q1[s:s + 1], kr[starts[s]:starts[s + 1]], v[starts[s]:starts[s + 1]], True, 0)
        packed_ref.check("o", o1[s:s + 1], one)
    assert cuda_api.device_status() == 0


def test_training_through_rotation_and_attention(cuda_api):
    """Gradients of a rotated packed attention with respect to the unrotated q and k: the inverse rotation of
    the attention's gradients, against the plain forms with the roundings of both steps."""
    lens = [90, 130]
    q, k, v, dout, starts, cu = _batch(lens, 8, 2, 64, 70, fused=True)
    pos = torch.randint(0, 300, (2, 220), generator=_gen(71), device="cuda").to(torch.int32)
    a = dict(rope_half_split=True, per_axis_freq=True)
    qr, kr = cuda_api.attn_rope_axes(q, k, pos, [16, 16], **a)
    o, lse = cuda_api.attn_packed_fwd(qr, kr, v, cu, causal=True)
    dq, dk, dv = cuda_api.attn_packed_bwd(qr, kr, v, o, lse, dout, cu, causal=True)
    cuda_api.attn_rope_axes(dq, dk, pos, [16, 16], inverse=True, q_out=dq, k_out=dk, **a)
    ref = packed_ref.packed(qr, kr, v, starts, True, 0, dout=dout)
    for name, got in (("dq", dq), ("dk", dk)):
        want, tol = packed_ref.rope_axes(ref[name], pos, [16, 16], False, True, True, 1e4, inverse=True)
        t = ref[name + "_tol"]
        pair = t[..., :32] + t[..., 32:]  # a rotation's output moves by at most the sum of its pair's errors
        tol = tol * (1 + packed_ref.U) + torch.cat([pair, pair], -1) * (1 + packed_ref.U)
        assert bool(((got.double() - want).abs() <= tol).all()), name


def test_other_stream_and_concurrent_calls(cuda_api):
    """Calls on two streams at once, each with its own workspace, equal the calls alone."""
    sets = [_batch(lens, 8, 2, 128, 80 + i) for i, lens in enumerate(([700, 3, 90], [50, 1200]))]
    alone = [cuda_api.attn_packed_fwd(q, k, v, cu, causal=True) for q, k, v, _, _, cu in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, (q, k, v, _, _, cu) in zip(streams, sets):
            s.wait_stream(torch.cuda.current_stream())
            got.append(cuda_api.attn_packed_fwd(q, k, v, cu, causal=True, stream=s))
        torch.cuda.synchronize()
        for (o, lse), (o2, lse2) in zip(alone, got):
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
    raw = cuda_api.attn_packed_fwd(*sets[0][:3], sets[0][5], causal=True, stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(raw[0], alone[0][0])


def test_graph_replays_with_other_lengths(cuda_api):
    """A captured training step and a captured chunk step, replayed after the offsets, lengths and inputs
    changed in place."""
    Hq, Hkv, D, T, S = 8, 2, 64, 300, 3
    q, k, v, dout, starts, cu = _batch([100, 100, 100], Hq, Hkv, D, 90)
    kp, vp, table = _cache([400, 400, 400], Hkv, D, 91)
    for x in (kp, vp):
        x.copy_(_randn(_gen(95), *x.shape))
    table_d = table.cuda()
    lens = torch.tensor([100, 200, 300], dtype=torch.int32, device="cuda")
    step = lambda: (cuda_api.attn_packed_fwd(q, k, v, cu, causal=True),)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True)
        grads = cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True)
        oc, lc = cuda_api.attn_chunk_paged(q, kp, vp, table_d, lens, cu, k_new=k, v_new=v)
    for i, new in enumerate(([100, 100, 100], [1, 298, 1], [0, 130, 170])):
        starts = [0, new[0], new[0] + new[1], T]
        cu.copy_(torch.tensor(starts, dtype=torch.int32))
        total = [n + 50 * i for n in new]
        lens.copy_(torch.tensor(total, dtype=torch.int32))
        q.copy_(_randn(_gen(92 + i), T, Hq, D))
        graph.replay()
        torch.cuda.synchronize()
        assert cuda_api.device_status() == 0
        ref = packed_ref.packed(q, k, v, starts, True, 0, dout=dout)
        for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + tuple(grads)):
            packed_ref.check(name, x, ref)
        for j, n in enumerate(new):
            if n:
                r = packed_ref.attend(q[starts[j]:starts[j + 1]], _rows(kp, table, j, total[j]),
                                      _rows(vp, table, j, total[j]), True, 0)
                packed_ref.check("o", oc[starts[j]:starts[j + 1]], r)


def test_empty_and_zero_tokens(cuda_api):
    q, k, v, dout, _, _ = _batch([5], 4, 2, 64, 96)
    cu = torch.tensor([2, 2, 2], dtype=torch.int32, device="cuda")
    o = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = cuda_api.attn_packed_fwd(q, k, v, cu, o=o)
    dq, dk, dv = (torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (q, k, v))
    cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in (o, dq, dk, dv)) and cuda_api.device_status() == 0
    e = [x[:0] for x in (q, k, v)]
    o0, lse0 = cuda_api.attn_packed_fwd(*e, cu * 0)
    assert o0.shape == (0, 4, 64) and lse0.shape == (4, 0)
    assert [x.shape[0] for x in cuda_api.attn_packed_bwd(*e, o0, lse0, o0, cu * 0)] == [0, 0, 0]
    y, _ = cuda_api.attn_rope_axes(e[0], e[1], torch.zeros(1, 0, dtype=torch.int32, device="cuda"), [32])
    assert y.shape == (0, 4, 64)


def test_binding_refusals_on_the_gpu(cuda_api):
    q, k, v, dout, _, cu = _batch([5], 4, 2, 64, 97)
    with pytest.raises(TypeError):
        cuda_api.attn_packed_fwd(q.float(), k, v, cu)
    with pytest.raises(TypeError):
        cuda_api.attn_packed_fwd(q, k, v, cu.long())
    with pytest.raises(ValueError):
        cuda_api.attn_packed_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, cu)
    with pytest.raises(ValueError):
        cuda_api.attn_packed_fwd(q, k, v, cu.cpu())
    with pytest.raises(cuda_api.AttnError):
        cuda_api.attn_packed_fwd(q, k, v, cu, causal=False, window=3)
    with pytest.raises(cuda_api.AttnError):
        cuda_api.attn_packed_fwd(q, k, v, cu, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    x = torch.zeros(5, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(cuda_api.AttnError):  # rows 520 bytes apart are not 16-byte aligned
        cuda_api.attn_packed_fwd(x[:, :256].view(5, 4, 64), k, v, cu)


@pytest.mark.parametrize("which", ["packed", "chunk", "backward"])
def test_timeout_is_reported_and_the_context_survives(cuda_api, which):
    """One copy of the first CTA never happens (test hook): the bounded wait runs out, the call ends with
    the status bit set, and the next call works."""
    q, k, v, dout, starts, cu = _batch([300, 20], 8, 2, 128, 98)
    kp, vp, table = _cache([300, 20], 2, 128, 99)
    lens = torch.tensor([300, 20], dtype=torch.int32, device="cuda")
    o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True)
    call = {"packed": lambda: cuda_api.attn_packed_fwd(q, k, v, cu, causal=True),
            "chunk": lambda: cuda_api.attn_chunk_paged(q, kp, vp, table.cuda(), lens, cu, k_new=k, v_new=v),
            "backward": lambda: cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True)}[which]
    assert cuda_api.device_status() == 0
    cuda_api.debug_drop_copy(True)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        cuda_api.debug_drop_copy(False)
    assert cuda_api.device_status() & cuda_api.DEVICE_TIMEOUT
    got = call()
    torch.cuda.synchronize()
    assert cuda_api.device_status() == 0
    ref = packed_ref.packed(q, k, v, starts, True, 0, dout=dout)
    if which == "backward":
        for name, x in zip(("dq", "dk", "dv"), got):
            packed_ref.check(name, x, ref)
    else:
        packed_ref.check("o", got[0], ref)


# ------------------------------------------------------------------ calls that are allowed and easy to forget
def test_gradients_into_one_fused_tensor(cuda_api):
    """dq, dk, dv as views of the gradient of a fused projection's output, whose other columns stay."""
    for Hq, Hkv, D in ((8, 2, 128), (6, 2, 64)):
        q, k, v, dout, starts, cu = _batch([70, 200, 1], Hq, Hkv, D, 101, before=2, after=3, fused=True)
        o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True)
        g = torch.full((q.shape[0], Hq + 2 * Hkv + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
        cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True, dq=g[:, :Hq], dk=g[:, Hq:Hq + Hkv],
                                 dv=g[:, Hq + Hkv:Hq + 2 * Hkv])
        ref = packed_ref.packed(q, k, v, starts, True, 0, dout=dout)
        for name, x in (("dq", g[:, :Hq]), ("dk", g[:, Hq:Hq + Hkv]), ("dv", g[:, Hq + Hkv:Hq + 2 * Hkv])):
            packed_ref.check(name, x, ref)
        assert bool((g[:, -1] == 7).all()) and bool((g[:2] == 7).all()) and bool((g[-3:] == 7).all())


def test_chunk_shared_pages(cuda_api):
    """Two sequences share the pages of a common beginning (one of them a page in two places of its row)."""
    kp, vp, table = _cache([64, 64], 2, 128, 102, spare=6, extra_blocks=6)
    shared = table[0, :4].clone()
    rows = torch.full((2, 8), -1, dtype=torch.int32)
    free = [p for p in range(kp.shape[0]) if p not in shared.tolist()]
    rows[0, :6] = torch.tensor(shared.tolist() + free[:2])
    rows[1, :7] = torch.tensor(shared.tolist() + [int(shared[1])] + free[2:4])
    new, total = [20, 30], [64 + 20, 80 + 30]
    q, kn, vn, _, starts, cu = _batch(new, 8, 2, 128, 103)
    o, lse = cuda_api.attn_chunk_paged(q, kp, vp, rows.cuda(), torch.tensor(total, dtype=torch.int32, device="cuda"), cu,
                                       k_new=kn, v_new=vn)
    assert cuda_api.device_status() == 0
    for s in range(2):
        a, b = starts[s], starts[s + 1]
        k_all, v_all = _rows(kp, rows, s, total[s]), _rows(vp, rows, s, total[s])
        assert torch.equal(k_all[-new[s]:], kn[a:b]) and torch.equal(v_all[-new[s]:], vn[a:b])
        ref = packed_ref.attend(q[a:b], k_all, v_all, True, 0)
        packed_ref.check("o", o[a:b], ref)
        packed_ref.check("lse", lse[a:b].t(), ref)


def test_chunk_many_sequences(cuda_api):
    """More sequences than the plan keeps in shared memory, one or no token each."""
    rng = random.Random(104)
    new = [rng.choice([0, 1, 1, 2]) for _ in range(2300)]
    ctx = [rng.choice([0, 3, 15, 16, 40]) for _ in new]
    ctx = [c if n or c else 1 for c, n in zip(ctx, new)]
    _check_chunk(cuda_api, ctx, new, 4, 2, 64, 0, seed=105)


def test_rows_beyond_32_bit_offsets(cuda_api):
    """A sequence at the end of tensors of more than 2^31 elements (and bytes of a gradient, a workspace)."""
    T, Hq, Hkv, D, n = 540_000, 32, 8, 128, 300
    g = _gen(106)
    q, dout = (torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (q, dout, k, v):
        x[T - n - 200:] = NAN
        x[T - n:] = _randn(g, n, *x.shape[1:])
    cu = torch.tensor([T - n, T], dtype=torch.int32, device="cuda")
    ref = packed_ref.attend(q[T - n:], k[T - n:], v[T - n:], True, 0, dout=dout[T - n:])
    o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True)
    packed_ref.check("o", o[T - n:], ref)
    packed_ref.check("lse", lse[:, T - n:], ref)
    for name, x in zip(("dq", "dk", "dv"), cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True)):
        packed_ref.check(name, x[T - n:], ref)
    pos = torch.zeros(1, T, dtype=torch.int32, device="cuda")
    pos[0, T - n:] = torch.arange(n, dtype=torch.int32, device="cuda")
    first = q[T - n:].clone()
    y, _ = cuda_api.attn_rope_axes(q, k, pos, [64], q_out=q, k_out=k)
    want, tol = packed_ref.rope_axes(first, pos[:, T - n:], [64], False, False, False, 1e4)
    assert bool(((y[T - n:].double() - want).abs() <= tol).all())
    assert cuda_api.device_status() == 0


def test_pages_beyond_32_bit_offsets(cuda_api):
    """Pages at the end of pools of more than 2^31 elements."""
    pool, Hkv, D, n, ctx = 140_000, 8, 128, 40, 500
    kp, vp = (torch.empty(pool, Hkv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = (ctx + n + 15) // 16
    table = torch.arange(pool - pages, pool, dtype=torch.int32).flip(0)[None].contiguous()
    g = _gen(107)
    for x in (kp, vp):
        x[pool - pages:] = _randn(g, pages, Hkv, 16, D)
    q, kn, vn, _, _, cu = _batch([n], 16, Hkv, D, 108)
    o, lse = cuda_api.attn_chunk_paged(q, kp, vp, table.cuda(), torch.tensor([ctx + n], dtype=torch.int32, device="cuda"),
                                       cu, k_new=kn, v_new=vn)
    assert cuda_api.device_status() == 0
    k_all, v_all = _rows(kp, table, 0, ctx + n), _rows(vp, table, 0, ctx + n)
    assert torch.equal(k_all[ctx:], kn) and torch.equal(v_all[ctx:], vn)
    packed_ref.check("o", o, packed_ref.attend(q, k_all, v_all, True, 0))


def test_backward_and_chunks_on_two_streams(cuda_api):
    """A training step and a serving step at once, on streams of their own, equal the calls alone."""
    q, k, v, dout, starts, cu = _batch([400, 90], 8, 2, 64, 109)
    kp, vp, table = _cache([900, 300], 2, 64, 110)
    new = [50, 1]
    qc, kn, vn, _, _, cuc = _batch(new, 8, 2, 64, 111)
    lens, table_d = torch.tensor([900, 300], dtype=torch.int32, device="cuda"), table.cuda()
    chunk = lambda s: cuda_api.attn_chunk_paged(qc, kp, vp, table_d, lens, cuc, k_new=kn, v_new=vn, stream=s)

    def train(s):
        o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True, stream=s)
        return (o, lse) + tuple(cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True, stream=s))

    alone = train(None), chunk(None)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ref = packed_ref.packed(q, k, v, starts, True, 0, dout=dout)
    for _ in range(4):
        for s in (s1, s2):
            s.wait_stream(torch.cuda.current_stream())
        a, b = train(s1), chunk(s2)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(b, alone[1]))
        for name, x, y in zip(("o", "lse", "dq", "dk", "dv"), a, alone[0]):
            packed_ref.check(name, x, ref)
            assert name == "dq" or torch.equal(x, y)  # (dq's order of summation is free)


# ------------------------------------------------------------------ alignment, values that are not finite, the work list
def _plan_items(ws, S):
    """The forward work list in a workspace: int32 [items, 8] (first query row, position, sequence or first key
    row, keys, first key tile, key tiles, tokens | part << 10 | (parts - 1) << 20, slot)."""
    w = ws.cpu()
    n = int(w[:4].view(torch.int32))
    at = 256 + ((S + 1) * 4 + 255) // 256 * 256
    return w[at:at + 32 * n].clone().view(torch.int32).view(n, 8)


def _at_16_modulo_32(shape, dtype, fill):
    """A tensor whose memory starts 16 bytes behind a 32-byte border."""
    n = 1
    for x in shape:
        n *= x
    raw = torch.empty(n + 64, dtype=dtype, device="cuda")
    size = raw.element_size()
    at = ((16 - raw.data_ptr()) % 32) // size
    x = raw[at:at + n].view(shape)
    assert x.data_ptr() % 32 == 16
    return x.fill_(fill)


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 128), (4, 4, 64), (6, 2, 64)])
def test_buffers_at_16_byte_borders(cuda_api, Hq, Hkv, D):
    """Workspace and outputs 16 bytes behind a 32-byte border: what the header asks for and no more, on calls
    that cut keys into parts (blocks of two query tiles, single tokens) and on one that cuts nothing."""
    ws = lambda n: _at_16_modulo_32((n,), torch.uint8, 0xff)
    out = lambda T: _at_16_modulo_32((T, Hq, D), torch.bfloat16, 7.0)
    for lens, cut in (([2500, 1, 3000], True), ([40, 130], False)):
        T, S = sum(lens), len(lens)
        q, k, v, dout, starts, cu = _batch(lens, Hq, Hkv, D, 120)
        w = ws(cuda_api.packed_fwd_workspace_size(T, S, Hq, Hkv, D))
        o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True, o=out(T), workspace=w)
        assert bool(((_plan_items(w, S)[:, 6] >> 20) > 0).any()) == cut
        ref = packed_ref.packed(q, k, v, starts, True, 0, dout=dout)
        packed_ref.check("o", o, ref)
        packed_ref.check("lse", lse, ref)
        w = ws(cuda_api.packed_bwd_workspace_size(T, S, Hq, Hkv, D))
        grads = [_at_16_modulo_32(x.shape, torch.bfloat16, 7.0) for x in (q, k, v)]
        cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True, dq=grads[0], dk=grads[1], dv=grads[2],
                                 workspace=w)
        for name, x in zip(("dq", "dk", "dv"), grads):
            packed_ref.check(name, x, ref)
    for new, total in (([1, 1], [9000, 700]), ([300, 2], [6000, 40])):
        kp, vp, table = _cache(total, Hkv, D, 121)
        q, kn, vn, _, starts, cu = _batch(new, Hq, Hkv, D, 122)
        w = ws(cuda_api.chunk_workspace_size(sum(new), 2, table.shape[1], 16, Hq, Hkv, D))
        o, lse = cuda_api.attn_chunk_paged(q, kp, vp, table.cuda(), torch.tensor(total, dtype=torch.int32, device="cuda"),
                                           cu, k_new=kn, v_new=vn, o=out(sum(new)), workspace=w)
        assert bool(((_plan_items(w, 2)[:, 6] >> 20) > 0).any())
        for s in range(2):
            a, b = starts[s], starts[s + 1]
            ref = packed_ref.attend(q[a:b], _rows(kp, table, s, total[s]), _rows(vp, table, s, total[s]), True, 0)
            packed_ref.check("o", o[a:b], ref)
            packed_ref.check("lse", lse[a:b].t(), ref)
    assert cuda_api.device_status() == 0


def _spoil(q, k, row):
    """Queries that are not finite: rows `row` to `row` + 3 of head 0 get a NaN, an infinity (scores of both
    signs), and an infinity of the sign that makes every score -inf (k[:, 0, 9] is positive)."""
    k[:, 0, 9] = k[:, 0, 9].abs() + 0.125
    q[row, 0, 3], q[row + 1, 0, 5], q[row + 2, 0, 7], q[row + 3, 0, 9] = NAN, float("inf"), -float("inf"), -float("inf")


def _check_spoiled(ref, o, lse, row, n):
    """o [n, Hq, D], lse [Hq, n] of one sequence: NaN in head 0 of the four rows (lse -inf where all scores
    are), everything else as the plain form says."""
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[row:row + 4] = True
    assert bool(torch.isnan(ref["o"][bad, 0]).all()) and bool(torch.isnan(o[bad, 0].float()).all())
    assert bool(torch.isnan(lse[0, row:row + 3]).all()) and lse[0, row + 3].item() == -float("inf")
    ref["lse"][0, bad] = NAN  # (compared above)
    packed_ref.check("o", o, ref)
    packed_ref.check("lse", lse, ref)


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 128), (4, 4, 64), (6, 2, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 700), (False, 0)])
def test_queries_that_are_not_finite(cuda_api, Hq, Hkv, D, causal, window):
    """A NaN or infinite query shows in its own row, whether its block's keys are cut into parts or not, and
    in every part."""
    for lens, row in (([2500, 3000], 5), ([2500, 3000], 2990), ([130, 90], 60)):
        q, k, v, _, starts, cu = _batch(lens, Hq, Hkv, D, 130)
        a = starts[1]
        _spoil(q[a:], k[a:], row)
        o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=causal, window=window)
        packed_ref.check("o", o[:a], packed_ref.attend(q[:a], k[:a], v[:a], causal, window))
        _check_spoiled(packed_ref.attend(q[a:], k[a:], v[a:], causal, window), o[a:], lse[:, a:], row, lens[1])
    assert cuda_api.device_status() == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("new,total", [([4], [9000]), ([400], [7000]), ([4], [60])])
def test_chunk_queries_that_are_not_finite(cuda_api, Hq, Hkv, D, new, total):
    kp, vp, table = _cache(total, Hkv, D, 131)
    q, kn, vn, _, _, cu = _batch(new, Hq, Hkv, D, 132)
    _spoil(q, kn, new[0] - 4)
    kp[:, 0, :, 9] = kp[:, 0, :, 9].abs() + 0.125
    o, lse = cuda_api.attn_chunk_paged(q, kp, vp, table.cuda(), torch.tensor(total, dtype=torch.int32, device="cuda"),
                                       cu, k_new=kn, v_new=vn)
    ref = packed_ref.attend(q, _rows(kp, table, 0, total[0]), _rows(vp, table, 0, total[0]), True, 0)
    _check_spoiled(ref, o, lse.t(), new[0] - 4, new[0])
    assert cuda_api.device_status() == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (6, 2, 64)])
def test_joined_parts_repeat_bit_for_bit(cuda_api, Hq, Hkv, D):
    """Single tokens and chunks whose keys are cut into many parts, joined by whichever warp is last, each time
    on a workspace that holds other calls' states."""
    new, total = [1, 40, 1, 3], [20000, 9000, 300, 16]
    kp, vp, table = _cache(total, Hkv, D, 133)
    q, kn, vn, _, starts, cu = _batch(new, Hq, Hkv, D, 134)
    lens, t = torch.tensor(total, dtype=torch.int32, device="cuda"), table.cuda()
    w = torch.empty(cuda_api.chunk_workspace_size(sum(new), 4, table.shape[1], 16, Hq, Hkv, D), dtype=torch.uint8,
                    device="cuda")
    first = cuda_api.attn_chunk_paged(q, kp, vp, t, lens, cu, k_new=kn, v_new=vn, workspace=w)
    assert int(_plan_items(w, 4)[:, 6].max() >> 20) >= 16  # parts - 1 of the longest
    for s in range(4):
        a, b = starts[s], starts[s + 1]
        ref = packed_ref.attend(q[a:b], _rows(kp, table, s, total[s]), _rows(vp, table, s, total[s]), True, 0)
        packed_ref.check("o", first[0][a:b], ref)
        packed_ref.check("lse", first[1][a:b].t(), ref)
    other = q.flip(0).contiguous()
    for _ in range(30):
        cuda_api.attn_chunk_paged(other, kp, vp, t, lens, cu, k_new=kn, v_new=vn, workspace=w)
        o, lse = cuda_api.attn_chunk_paged(q, kp, vp, t, lens, cu, k_new=kn, v_new=vn, workspace=w)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    assert cuda_api.device_status() == 0


def test_a_stream_of_another_device_is_refused(cuda_api):
    q, k, v, dout, _, cu = _batch([5], 4, 2, 64, 135)
    kp, vp, table = _cache([5], 2, 64, 136)
    lens = torch.tensor([5], dtype=torch.int32, device="cuda")
    o, lse = cuda_api.attn_packed_fwd(q, k, v, cu)
    pos = torch.zeros(1, 5, dtype=torch.int32, device="cuda")
    here, there = torch.cuda.Stream(), q.get_device() + 1
    calls = [lambda s: cuda_api.attn_packed_fwd(q, k, v, cu, stream=s),
             lambda s: cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, stream=s),
             lambda s: cuda_api.attn_chunk_paged(q, kp, vp, table.cuda(), lens, cu, k_new=k, v_new=v, stream=s),
             lambda s: cuda_api.attn_rope_axes(q, k, pos, [32], stream=s)]
    for call in calls:
        with pytest.raises(ValueError, match="stream"):
            call(types.SimpleNamespace(cuda_stream=here.cuda_stream, device=torch.device("cuda", there)))
        call(types.SimpleNamespace(cuda_stream=here.cuda_stream, device=q.device))
    torch.cuda.synchronize()
    assert cuda_api.device_status() == 0


def test_windows_past_32_bits(cuda_api):
    q, k, v, dout, starts, cu = _batch([300, 20], 4, 2, 64, 137)
    kp, vp, table = _cache([300, 20], 2, 64, 138)
    lens = torch.tensor([300, 20], dtype=torch.int32, device="cuda")
    run = lambda w: cuda_api.attn_packed_fwd(q, k, v, cu, causal=True, window=w) + \
        cuda_api.attn_chunk_paged(q, kp, vp, table.cuda(), lens, cu, k_new=k, v_new=v, window=w)
    o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True)
    ref = packed_ref.packed(q, k, v, starts, True, 0, dout=dout)
    want = run(0)
    for w in (2 ** 32 + 5, -2 ** 32 + 5, 2 ** 31):
        assert all(torch.equal(x, y) for x, y in zip(run(w), want))
        for name, x in zip(("dq", "dk", "dv"), cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True, window=w)):
            packed_ref.check(name, x, ref)
    assert cuda_api.device_status() == 0


def _expected_list(new, keys, TT, Hkv, causal, window, starts, paged):
    """The rule of the forward's work list, restated: the blocks (first row, position, sequence or first key row,
    keys, first tile, tiles, tokens), their costs, the limit, and whether the list is cut."""
    blocks = []
    for s, (n, m) in enumerate(zip(new, keys)):
        for first in range(0, n, 2 * TT):
            tok = min(2 * TT, n - first)
            pos = m - n + first
            lo = max(0, pos - window + 1) if window > 0 else 0
            hi = pos + tok if causal else m
            jb = lo // 128
            tiles = (hi + 127) // 128 - jb
            blocks.append((starts[s] + first, pos, s if paged else starts[s], m, jb, tiles, tok))
    cost = lambda tiles, tok: (5 * tiles + 7) // 8 if tok <= TT else tiles
    costs = [cost(b[5], b[6]) for b in blocks]
    limit, longest = max(4, -(-sum(costs) * Hkv // 296)), max(costs)

    def load(cut):
        """The sum of every 148th item of the descending list, in steps of the counting sort's buckets."""
        hist = [0] * 1024
        for b, c in zip(blocks, costs):
            parts = -(-c // limit) if cut and c > limit else 1
            for i in range(parts):
                t = b[5] // parts + (i < b[5] % parts)
                hist[1023 - cost(t, b[6]) * 1023 // longest] += 1
        at = total = 0
        for i, n in enumerate(hist):
            if n:
                total += (-(-(at + n) * Hkv // 148) - -(-at * Hkv // 148)) * -(-(1023 - i) * longest // 1023)
            at += n
        return total

    join = 6 if any(c > limit and 4 * b[6] > TT for b, c in zip(blocks, costs)) else 2
    return blocks, costs, cost, limit, longest, longest > limit and load(True) + join < load(False)


def _check_list(ws, S, expected):
    blocks, costs, cost, limit, longest, cut = expected
    want = set()
    for b, c in zip(blocks, costs):
        parts = -(-c // limit) if cut and c > limit else 1
        at = b[4]
        for i in range(parts):
            t = b[5] // parts + (i < b[5] % parts)
            want.add(b[:4] + (at, t, b[6] | i << 10 | (parts - 1) << 20))
            at += t
    items = _plan_items(ws, S).tolist()
    assert len(items) == len(want) and {tuple(x[:7]) for x in items} == want
    order = [cost(x[5], x[6] & 1023) * 1023 // longest for x in items]
    assert order == sorted(order, reverse=True)
    taken = [r for slot, p in {(x[7], (x[6] >> 20) + 1) for x in items if x[6] >> 20} for r in range(slot, slot + p)]
    assert sorted(taken) == list(range(len(taken)))  # every slot is one part's
    return cut


def test_work_list_is_the_rule_s(cuda_api):
    """The list that the device builds: every block's tiles once, longest first, cut where the rule says so."""
    rng = random.Random(140)
    cuts = []
    for Hq, Hkv, causal, window in ((8, 2, True, 0), (4, 4, False, 0), (6, 2, True, 300), (8, 1, True, 0), (64, 1, True, 0)):
        for lens in ([1500], [2500, 1, 3000], [rng.randint(0, 400) for _ in range(40)], [1] * 5,
                     [rng.choice([0, 1, 2, 150]) for _ in range(2300)]):
            q, k, v, _, starts, cu = _batch(lens, Hq, Hkv, 64, 141)
            w = torch.empty(cuda_api.packed_fwd_workspace_size(sum(lens), len(lens), Hq, Hkv, 64), dtype=torch.uint8,
                            device="cuda")
            cuda_api.attn_packed_fwd(q, k, v, cu, causal=causal, window=window, workspace=w)
            cuts.append(_check_list(w, len(lens), _expected_list(lens, lens, 128 // (Hq // Hkv), Hkv, causal, window,
                                                                 starts, False)))
        for new, ctx in (([1] * 8, [4000] * 8), ([1, 300, 1, 0, 20], [9000, 2000, 3, 77, 500]), ([1], [2000]),
                         ([1] * 200, [rng.randint(0, 900) for _ in range(200)])):
            if not causal:
                continue
            total = [c + n for c, n in zip(ctx, new)]
            kp, vp, table = _cache(total, Hkv, 64, 142)
            q, kn, vn, _, starts, cu = _batch(new, Hq, Hkv, 64, 143)
            w = torch.empty(cuda_api.chunk_workspace_size(sum(new), len(new), table.shape[1], 16, Hq, Hkv, 64),
                            dtype=torch.uint8, device="cuda")
            cuda_api.attn_chunk_paged(q, kp, vp, table.cuda(), torch.tensor(total, dtype=torch.int32, device="cuda"),
                                      cu, k_new=kn, v_new=vn, window=window, workspace=w)
            cuts.append(_check_list(w, len(new), _expected_list(new, total, 128 // (Hq // Hkv), Hkv, True, window,
                                                                starts, True)))
    assert any(cuts) and not all(cuts)
    assert cuda_api.device_status() == 0


def test_backward_tile_list(cuda_api):
    """The backward's list: every 128 keys of every sequence once, a sequence's tiles in their order, sequences
    from the longest to the shortest (to the 1,023rd part of the longest), query tiles numbered through."""
    rng = random.Random(144)
    for Hq, Hkv in ((8, 2), (6, 2), (4, 4)):
        TT = 128 // (Hq // Hkv)
        for lens in ([700], [1, 0, 300, 128, 129, 0, 2000, 5], [rng.choice([0, 1, 2, 150, 300]) for _ in range(2300)]):
            S, T = len(lens), sum(lens)
            q, k, v, dout, starts, cu = _batch(lens, Hq, Hkv, 64, 145)
            w = torch.empty(cuda_api.packed_bwd_workspace_size(T, S, Hq, Hkv, 64), dtype=torch.uint8, device="cuda")
            o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True)
            cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True, workspace=w)
            up = lambda x: (x + 255) // 256 * 256
            at = 256 + up((S + 1) * 4) + 2 * up(S * 4)
            n_max = T // 128 + min(S, T)
            want, base = [], 0
            for s, n in enumerate(lens):
                want += [[starts[s], n, t, base] for t in range((n + 127) // 128)]
                base += -(-n // TT)
            n = int(w[:4].cpu().view(torch.int32))
            tiles = w[at:at + 16 * n].cpu().clone().view(torch.int32).view(n, 4).tolist()
            assert tiles == want
            at += up(16 * n_max)
            order = w[at:at + 4 * n].cpu().clone().view(torch.int32).tolist()
            assert sorted(order) == list(range(n))
            most = max((x + 127) // 128 for x in lens)
            left = [((x[1] + 127) // 128 * 1023 // most, x[0], x[2]) for x in (want[i] for i in order)]
            heads = [x for x in left if x[2] == 0]
            assert [x[0] for x in heads] == sorted((x[0] for x in heads), reverse=True)
            for a, b in zip(left, left[1:]):
                assert b[2] == 0 or (b[1] == a[1] and b[2] == a[2] + 1)
    assert cuda_api.device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_backward_of_a_query_that_is_not_finite(cuda_api, D):
    """One NaN and one infinite query among finite ones: their own dq is NaN, every other row's dq is right (it
    takes part in no other row's sum), and so are the gradients of the other sequences."""
    q, k, v, dout, starts, cu = _batch([150, 600, 90], 8, 2, D, 146)
    q[200, 0, 3], q[500, 5, 7] = NAN, float("inf")
    o, lse = cuda_api.attn_packed_fwd(q, k, v, cu, causal=True)
    grads = cuda_api.attn_packed_bwd(q, k, v, o, lse, dout, cu, causal=True)
    ref = packed_ref.packed(q, k, v, starts, True, 0, dout=dout)
    bad = torch.zeros(q.shape[0], 8, dtype=torch.bool, device="cuda")
    bad[200, 0] = bad[500, 5] = True
    assert bool(torch.isnan(grads[0][bad].float()).all())
    ref["dq"][bad] = NAN  # (compared above)
    packed_ref.check("dq", grads[0], ref)
    for name, x in zip(("dk", "dv"), grads[1:]):
        for a, b in ((0, 150), (750, 840)):
            packed_ref.check(name, x[a:b], {n: y[a:b] for n, y in ref.items() if n.startswith(name)})
    assert cuda_api.device_status() == 0
