"""The operators on packed sequences on the CPU: the index arithmetic of the work list against brute
force, refusals before any CUDA call, and the gradients of the tests' plain form against differences."""
import ctypes
import os
import subprocess
import types

import pytest
import torch

import packed_ref
from exact_attention_161_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def api():
    build.build()
    from exact_attention_161_b200 import api as api_mod
    return api_mod


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """csrc/plan.cuh compiled for the host."""
    d = tmp_path_factory.mktemp("plan")
    src = d / "plan.cpp"
    src.write_text('#include "plan.cuh"\nusing namespace attn;\nextern "C" {\n'
                   'void keys(int f, int l, int m, int c, int w, int* o) { KeyTiles t = key_tiles(f, l, m, c, w);'
                   ' o[0] = t.jb; o[1] = t.n; }\n'
                   'void queries(int t, int n, int q, int c, int w, int* o) { query_tiles(t, n, q, c, w, o[0], o[1]); }\n'
                   'int limit(long long t, int h) { return plan_limit(t, h); }\n'
                   'int parts(int t, int l) { return plan_parts(t, l); }\n'
                   'void part(int t, int p, int i, int* o) { plan_part(t, p, i, o[0], o[1]); }\n'
                   'long long slots(long long T, long long S, int TT, long long m, int h)'
                   ' { return plan_layout(T, S, TT, m, h, 128).max_slots; }\n'
                   'long long items(long long T, long long S, int TT, long long m, int h)'
                   ' { return plan_layout(T, S, TT, m, h, 128).max_items; }\n'
                   'long long tiles(long long T, long long S) { return bwd_plan_layout(T, S, 128, 1, 64).max_tiles; }\n'
                   'long long q_tiles(long long T, long long S, int TT)'
                   ' { return bwd_plan_layout(T, S, TT, 1, 64).max_q_tiles; }\n'
                   'int meta(int n, int p, int q) { PackedItem x; x.meta = make_meta(n, p, q);'
                   ' return item_tokens(x) == n && item_part(x) == p && item_parts(x) == q; }\n}\n')
    lib = d / "libplan.so"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "exact_attention_161_b200", "csrc"), str(src), "-o", str(lib)], check=True)
    p = ctypes.CDLL(str(lib))
    for f, n in ((p.slots, 5), (p.items, 5), (p.tiles, 2), (p.q_tiles, 3)):
        f.restype = ctypes.c_longlong
        f.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong, ctypes.c_int][:n]
    p.limit.argtypes = [ctypes.c_longlong, ctypes.c_int]
    return p


def _pair(fn, *args):
    o = (ctypes.c_int * 2)()
    fn(*args, o)
    return o[0], o[1]


@pytest.mark.parametrize("causal,window", [(1, 0), (0, 0), (1, 1), (1, 2), (1, 127), (1, 128), (1, 129), (1, 300),
                                           (1, 2147483647)])
def test_visible_tiles_against_brute_force(plan, causal, window):
    def sees(i, j, m):
        return j < m and (not causal or j <= i) and (window == 0 or j > i - window)

    for n, m in [(1, 1), (1, 700), (5, 130), (127, 127), (128, 128), (129, 129), (300, 300), (64, 513), (200, 1000)]:
        off = m - n
        for first in range(0, n, 37):
            for size in (1, 31, 64):
                last = min(n, first + size) - 1
                tiles = {j // 128 for j in range(m) if any(sees(off + i, j, m) for i in range(first, last + 1))}
                jb, cnt = _pair(plan.keys, off + first, off + last, m, causal, window)
                assert set(range(jb, jb + cnt)) == tiles, (n, m, first, last)
    for n, TT in [(1, 128), (100, 128), (128, 32), (129, 42), (500, 128), (500, 32), (500, 25), (300, 1), (1000, 64)]:
        for t in range((n + 127) // 128):
            tiles = {i // TT for i in range(n) for j in range(t * 128, min(n, t * 128 + 128)) if sees(i, j, n)}
            ib, ie = _pair(plan.queries, t, n, TT, causal, window)
            assert set(range(ib, ie)) == tiles, (n, t, TT)


@pytest.mark.parametrize("Hkv", [1, 2, 8, 32])
@pytest.mark.parametrize("TT", [1, 32, 42, 128])
def test_work_list_fits_the_workspace(plan, TT, Hkv):
    """Blocks, parts and slots of many length distributions against the sizes the layout reserves; the parts
    of a block cover its tiles once."""
    g = torch.Generator().manual_seed(TT * 100 + Hkv)
    for trial in range(40):
        S = int(torch.randint(1, 70, (1,), generator=g))
        top = int(10 ** (torch.rand(1, generator=g).item() * 4.5))
        new = torch.randint(0, max(2, top // (1 + trial % 7)), (S,), generator=g).tolist()
        ctx = torch.randint(0, top + 1, (S,), generator=g).tolist() if trial % 2 else [0] * S
        T = sum(new)
        if T == 0:
            continue
        max_keys = max(c + n for c, n in zip(ctx, new))
        if trial % 2 == 0:
            max_keys = T  # packed: a sequence may hold every token
        blocks, tiles_bwd, q_tiles = [], 0, 0
        for c, n in zip(ctx, new):
            tiles_bwd += -(-n // 128)
            q_tiles += -(-n // TT)
            for first in range(0, n, 2 * TT):
                last = min(n, first + 2 * TT) - 1
                blocks.append(_pair(plan.keys, c + first, c + last, c + n, 1, 0)[1])
        limit = plan.limit(sum(blocks), Hkv)
        slots = items = 0
        for t in blocks:
            p = plan.parts(t, limit)
            assert 1 <= p <= 1023 and plan.meta(2 * TT, p - 1, p)
            edges = [_pair(plan.part, t, p, i) for i in range(p)]
            assert edges[0][0] == 0 and edges[-1][1] == t and all(a[1] == b[0] for a, b in zip(edges, edges[1:]))
            assert all(b > a for a, b in edges)
            items += p
            slots += p if p > 1 else 0
        assert slots <= plan.slots(T, S, TT, max_keys, Hkv)
        assert items <= plan.items(T, S, TT, max_keys, Hkv)
        assert tiles_bwd <= plan.tiles(T, S) and q_tiles <= plan.q_tiles(T, S, TT)


FAKE, MISALIGNED = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)


def _fwd(api, q=FAKE, k=FAKE, v=FAKE, o=FAKE, cu=FAKE, lse=None, T=100, S=3, Hq=8, Hkv=2, D=128, causal=1, window=0,
         scale=0.0, qs=None, ks=None, ws=FAKE, ws_bytes=None):
    ws_bytes = api.packed_fwd_workspace_size(T, S, Hq, Hkv, D) if ws_bytes is None else ws_bytes
    return api.lib.attn_packed_fwd(q, k, v, Hq * D if qs is None else qs, Hkv * D if ks is None else ks, Hkv * D, cu, S,
                                   T, Hq, Hkv, D, causal, window, scale, o, lse, ws, ws_bytes, None)


SHARED = [
    (dict(q=None), 1), (dict(k=MISALIGNED), 1), (dict(cu=None), 1), (dict(cu=ctypes.c_void_p(0x10002)), 1),
    (dict(T=-1), 1), (dict(S=0), 1), (dict(Hq=3), 1), (dict(causal=2), 1), (dict(causal=0, window=4), 1),
    (dict(scale=float("nan")), 1), (dict(qs=1016), 1), (dict(qs=1028), 1), (dict(ws=None), 1), (dict(ws_bytes=16), 1),
    (dict(D=96), 2), (dict(Hq=129, Hkv=1), 2), (dict(T=1 << 30), 2), (dict(S=1 << 24), 2),
    (dict(T=(1 << 30) - 1, Hq=8), 2),
]


@pytest.mark.parametrize("kw,expect", SHARED + [(dict(o=None), 1), (dict(o=MISALIGNED), 1), (dict(ks=128), 1),
                                                (dict(lse=ctypes.c_void_p(0x10002)), 1)])
def test_packed_fwd_refusals(api, kw, expect):
    assert _fwd(api, **kw) == expect
    assert api.last_error() != ""


def _bwd(api, q=FAKE, k=FAKE, lse=FAKE, dout=FAKE, dq=FAKE, dk=FAKE, cu=FAKE, T=100, S=3, Hq=8, Hkv=2, D=128, causal=1,
         window=0, scale=0.0, qs=None, dks=None, ws=FAKE, ws_bytes=None):
    ws_bytes = api.packed_bwd_workspace_size(T, S, Hq, Hkv, D) if ws_bytes is None else ws_bytes
    return api.lib.attn_packed_bwd(q, k, FAKE, Hq * D if qs is None else qs, Hkv * D, Hkv * D, FAKE, lse, dout, dq, dk,
                                   FAKE, Hq * D, Hkv * D if dks is None else dks, Hkv * D, cu, S, T, Hq, Hkv, D, causal,
                                   window, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", SHARED + [(dict(lse=None), 1), (dict(dout=MISALIGNED), 1), (dict(dq=None), 1),
                                                (dict(dk=MISALIGNED), 1), (dict(dks=260), 1)])
def test_packed_bwd_refusals(api, kw, expect):
    assert _bwd(api, **kw) == expect
    assert api.last_error() != ""


def _chunk(api, q=FAKE, kn=FAKE, vn=FAKE, ks=None, kp=FAKE, bt=FAKE, lens=FAKE, cu=FAKE, T=100, S=3, max_blocks=8,
           pages=30, page=16, Hq=8, Hkv=2, D=128, window=0, scale=0.0, ws_bytes=None):
    ws_bytes = api.chunk_workspace_size(T, S, max_blocks, page, Hq, Hkv, D) if ws_bytes is None else ws_bytes
    return api.lib.attn_chunk_paged(q, kn, vn, Hq * D, Hkv * D if ks is None else ks, Hkv * D, kp, FAKE, bt, lens, cu, S,
                                    T, max_blocks, pages, page, Hq, Hkv, D, window, scale, FAKE, None, FAKE, ws_bytes,
                                    None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), 1), (dict(kn=None), 1), (dict(vn=None), 1), (dict(kn=MISALIGNED), 1), (dict(ks=128), 1),
    (dict(kp=None), 1), (dict(kp=MISALIGNED), 1), (dict(bt=ctypes.c_void_p(0x10002)), 1), (dict(lens=None), 1),
    (dict(cu=None), 1), (dict(pages=0), 1), (dict(max_blocks=0), 1), (dict(Hq=9), 1), (dict(ws_bytes=0), 1),
    (dict(scale=float("inf")), 1), (dict(page=32), 2), (dict(D=80), 2), (dict(max_blocks=1 << 26), 2),
    (dict(pages=1 << 30), 2),
])
def test_chunk_refusals(api, kw, expect):
    assert _chunk(api, **kw) == expect
    assert api.last_error() != ""


def _rope(api, q=FAKE, qo=FAKE, k=FAKE, ko=FAKE, pos=FAKE, T=10, Hq=4, Hk=2, D=128, sections=(16, 24, 24), inter=0,
          ladder=0, half=1, base=1e4, ps=1.0, inv=0, qs=None):
    sec = (ctypes.c_int * max(1, len(sections)))(*sections)
    return api.lib.attn_rope_axes(q, qo, k, ko, Hq * D if qs is None else qs, Hq * D, Hk * D, Hk * D, pos, T, Hq, Hk, D,
                                  len(sections), sec, inter, ladder, half, base, ps, inv, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(ko=MISALIGNED), 1), (dict(pos=None), 1),
    (dict(pos=ctypes.c_void_p(0x10001)), 1), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hk=-1), 1), (dict(sections=()), 1),
    (dict(sections=(0, 64)), 1), (dict(sections=(65,)), 1), (dict(sections=(32, 40)), 1), (dict(half=2), 1),
    (dict(inter=-1), 1), (dict(inv=3), 1), (dict(base=0.0), 1), (dict(ps=float("inf")), 1), (dict(qs=504), 1),
    (dict(sections=(8, 28, 28), inter=1), 1),  # axes 1 and 2 would need every other pair
    (dict(sections=(4, 4, 5)), 2), (dict(D=96), 2), (dict(sections=(8,) * 9), 2), (dict(T=1 << 30), 2),
    (dict(Hq=40000), 2),
])
def test_rope_axes_refusals(api, kw, expect):
    assert _rope(api, **kw) == expect
    assert api.last_error() != ""


def test_no_tokens_is_valid(api):
    """T = 0 returns before any pointer is looked at or any CUDA call is made."""
    assert _fwd(api, T=0, q=None, ws=None) == 0 and _bwd(api, T=0, q=None, ws=None) == 0
    assert _chunk(api, T=0, q=None) == 0 and _rope(api, T=0, q=None, pos=None) == 0


def test_workspace_sizes(api):
    # one short prompt: offsets, one block of at most four key tiles, nothing cut
    assert api.packed_fwd_workspace_size(10, 1, 8, 2, 128) == 256 + 256 + 256
    # partial states are bounded by the parts the split rule can make, however long the call
    assert api.packed_fwd_workspace_size(1 << 20, 4, 32, 8, 128) < 100 << 20
    assert api.chunk_workspace_size(64, 64, 1024, 16, 32, 8, 128) < 100 << 20
    # backward: per padded row and head two fp32 vectors and D fp32 sums
    # (128 tokens of 4 heads on 2 K/V heads: two tiles of 64 tokens, and one for the sequence's end)
    assert api.packed_bwd_workspace_size(128, 1, 4, 2, 128) == 6 * 256 + 3 * 2 * 128 * (2 + 128) * 4
    for bad in ((0, 1, 8, 2, 128), (10, 0, 8, 2, 128), (10, 1, 8, 3, 128), (10, 1, 256, 1, 128)):
        assert api.packed_fwd_workspace_size(*bad) == 0
    assert api.packed_bwd_workspace_size(10, 0, 8, 2, 128) == 0 and api.packed_bwd_workspace_size(9, 1, 8, 3, 128) == 0 and api.chunk_workspace_size(1, 1, 0, 16, 8, 2, 128) == 0


def test_binding_refuses_what_is_not_on_the_gpu(api):
    q, k = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        api.attn_rope_axes(q, k, torch.zeros(1, 4, dtype=torch.int32), [64], q_out=q, k_out=k, stream=0)
    with pytest.raises(ValueError):
        api.attn_packed_fwd(q, k[:3], k[:3], cu)
    with pytest.raises(ValueError):
        api.attn_packed_fwd(q, k, k, cu[:1])
    with pytest.raises(ValueError):
        api.attn_rope_axes(q, k, torch.zeros(2, 4, dtype=torch.int32), [64])
    with pytest.raises(ValueError):
        api.attn_chunk_paged(q, k[:, :, None], k[:, :, None], torch.zeros(2, 3, dtype=torch.int32), cu[1:], cu)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3)])
def test_plain_gradients_against_differences(causal, window):
    """The plain form that the GPU tests compare with: its gradients against central differences of its own
    forward in fp64 (step 1e-5: truncation below 1e-9, rounding below 1e-9)."""
    g = torch.Generator().manual_seed(5)
    q, k, v, w = (torch.randn(7, h, 4, generator=g, dtype=torch.float64) for h in (4, 2, 2, 4))
    starts = [0, 3, 3, 7]
    ref = packed_ref.packed(q, k, v, starts, causal, window, dout=w)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for _ in range(12):
            at = tuple(int(torch.randint(0, s, (1,), generator=g)) for s in x.shape)
            x0, vals = x[at].item(), []
            for h in (1e-5, -1e-5):
                x[at] = x0 + h
                vals.append((packed_ref.packed(q, k, v, starts, causal, window)["o"] * w).sum().item())
            x[at] = x0
            assert abs((vals[0] - vals[1]) / 2e-5 - ref[name][at].item()) < 1e-7


def test_plain_rotation_is_undone_by_its_inverse():
    g = torch.Generator().manual_seed(6)
    x = torch.randn(5, 3, 64, generator=g, dtype=torch.float64)
    pos = torch.randint(-1000, 1000, (3, 5), generator=g)
    for inter, ladder, half in ((False, False, True), (True, True, False)):
        a = (pos, [10, 7, 7], inter, ladder, half, 1e4, 2.0)
        y, _ = packed_ref.rope_axes(x, *a)
        z, _ = packed_ref.rope_axes(y, *a, inverse=True)
        assert (z - x).abs().max() < 1e-12 and (y - x).abs().max() > 0.1


def test_a_stream_of_another_device_is_refused(api):
    """Running there would hand one device's memory to another's kernels."""
    other = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        api._on(0, other, lambda st: pytest.fail("called"))


def test_numbers_past_32_bits_are_not_cut_off(api):
    """The C entry points take 32-bit integers, of which ctypes would pass the low bits: a window that long cuts
    nothing, a section that long is refused."""
    for window, passed in ((5, 5), (0, 0), (-3, -1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                           (2 ** 32 + 5, 2 ** 31 - 1), (-2 ** 32 + 5, -1)):
        assert ctypes.c_int(api._window(window)).value == passed
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    for sections in ([2 ** 32 + 64], [-2 ** 32 + 64]):
        with pytest.raises(ValueError, match="sections"):
            api.attn_rope_axes(q, None, torch.zeros(1, 4, dtype=torch.int32), sections)


@pytest.fixture(scope="module")
def costs(tmp_path_factory):
    """What the work list is cut by, compiled for the host."""
    d = tmp_path_factory.mktemp("costs")
    src = d / "costs.cpp"
    src.write_text('#include "plan.cuh"\nusing namespace attn;\nextern "C" {\n'
                   'void keys(int f, int l, int m, int c, int w, int* o) { KeyTiles t = key_tiles(f, l, m, c, w);'
                   ' o[0] = t.jb; o[1] = t.n; }\n'
                   'int cost(int t, int one) { return plan_cost(t, one); }\n'
                   'int limit(long long t, int h) { return plan_limit(t, h); }\n'
                   'int parts(int t, int l) { return plan_parts(t, l); }\n'
                   'void part(int t, int p, int i, int* o) { plan_part(t, p, i, o[0], o[1]); }\n'
                   'void sizes(long long T, long long S, int TT, long long m, int h, long long* o)'
                   ' { PlanLayout L = plan_layout(T, S, TT, m, h, 128); o[0] = L.max_slots; o[1] = L.max_items; }\n}\n')
    lib = d / "libcosts.so"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "exact_attention_161_b200", "csrc"), str(src), "-o", str(lib)], check=True)
    p = ctypes.CDLL(str(lib))
    p.limit.argtypes = [ctypes.c_longlong, ctypes.c_int]
    p.sizes.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong, ctypes.c_int,
                        ctypes.POINTER(ctypes.c_longlong)]
    return p


@pytest.mark.parametrize("Hkv", [1, 2, 8, 32])
@pytest.mark.parametrize("TT", [1, 16, 32, 42, 128])
@pytest.mark.parametrize("causal,window", [(1, 0), (0, 0), (1, 1), (1, 700)])
def test_list_cut_by_cost_fits_the_workspace(costs, TT, Hkv, causal, window):
    """The device's rule: blocks are cut by what they cost (5/8 of its tiles for a block of at most TT tokens), in
    calls of single tokens, of short chunks among full blocks, and of whole prompts. Items and slots stay within
    what the layout reserves, no part is empty, and the parts cover the block's tiles once."""
    g = torch.Generator().manual_seed(TT * 1000 + Hkv * 10 + causal + window)
    draw = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    for trial in range(20):
        S = draw(1, 70)
        top = int(10 ** (torch.rand(1, generator=g).item() * 4.5)) + 1
        kind = trial % 4
        ctx = [draw(0, top) for _ in range(S)]
        if trial == 0:  # one token on a long context: always cut, without a window
            new, ctx = [1], [60000]
        elif kind == 0:  # a token each
            new = [1] * S
        elif kind == 1:  # short chunks
            new = [draw(0, 2 * TT) for _ in range(S)]
        elif kind == 2:  # single tokens beside chunks
            new = [1 if draw(0, 3) else draw(1, 3000) for _ in range(S)]
        else:  # packed prompts
            new, ctx = [draw(0, top) for _ in range(S)], [0] * S
        S, T = len(new), sum(new)
        if T == 0:
            continue
        max_keys = T if kind == 3 else (max(c + n for c, n in zip(ctx, new)) + 15) // 16 * 16
        blocks = []
        for c, n in zip(ctx, new):
            for first in range(0, n, 2 * TT):
                last = min(n, first + 2 * TT) - 1
                tiles = _pair(costs.keys, c + first, c + last, c + n, causal, window)[1]
                one = int(last - first + 1 <= TT)
                cost = costs.cost(tiles, one)
                assert 1 <= cost <= tiles and cost >= tiles / 2
                blocks.append((tiles, cost, one))
        limit = costs.limit(sum(x[1] for x in blocks), Hkv)
        slots = items = 0
        for tiles, cost, one in blocks:
            p = costs.parts(cost, limit)
            assert 1 <= p <= 1023 and (p == 1) == (cost <= limit)
            edges = [_pair(costs.part, tiles, p, i) for i in range(p)]
            assert edges[0][0] == 0 and edges[-1][1] == tiles and all(a[1] == b[0] for a, b in zip(edges, edges[1:]))
            assert all(b > a for a, b in edges)
            items += p
            slots += p if p > 1 else 0
            assert trial > 0 or window > 0 or p > 1
        room = (ctypes.c_longlong * 2)()
        costs.sizes(T, S, TT, max_keys, Hkv, room)
        assert slots <= room[0] and items <= room[1]
