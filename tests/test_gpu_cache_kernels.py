"""The cache attention where one kernel hands over to another, where masks,
infinities and NaN meet the tensor cores, and where offsets pass 32 bits; whole
prompts in pieces; graphs that share a workspace."""
import numpy as np
import pytest
import torch

import block_sparse_attention_band_b200 as pb
from tests import cache_ref as R
from tests.test_gpu_cache import DEV, Planned, attn_case, check_attn, i32, no_error, run_attn

pytestmark = pytest.mark.gpu


# rows = new tokens x group: 16 | 17 .. 32 a unit, two units up to 64, then tiles of 128 in pairs
@pytest.mark.parametrize("group,add", [(1, 16), (1, 17), (4, 8), (3, 11), (4, 16), (5, 13), (13, 5), (4, 32), (3, 43),
                                       (4, 64), (1, 257), (64, 2), (2, 130)])
def test_rows_at_the_borders_between_kernels(group, add):
    lens, adds = [add + 300, add, add + 1000], [add, add, 1]
    c = attn_case(group * 1000 + add, lens, adds, 32, 2 * group, 2, spare=2)
    check_attn(c, run_attn(c, add))
    no_error()


@pytest.mark.parametrize("max_add", [90, 1])
def test_single_tokens_drafts_and_pieces_in_one_call(max_add):
    lens = [500, 1, 0, 90, 777, 130, 64, 2000, 33]
    adds = [1, 1, 0, 90, 5, 70, 17, 1, 33]
    c = attn_case(4, lens, adds, 16, 8, 2, spare=4)
    check_attn(c, run_attn(c, max_add))
    no_error()


def uneven_mask(c, hq, hkv, seed):
    """Masks as different as they get: all, none, one head alone, the first blocks, the last, odd ones; bits behind the
    tokens' blocks set at random."""
    rng = np.random.default_rng(seed)
    n, words = len(c["lens"]), (-(-c["wide"] * c["page"] // 128) + 31) // 32
    keep = np.zeros((n, hq, words * 32), bool)
    for i in range(n):
        blocks = -(-int(c["lens"][i]) // 128)
        for h in range(hq):
            kind = (i + h // (hq // hkv)) % 6
            if kind == 0:
                keep[i, h, :blocks] = True
            elif kind == 2:
                keep[i, h, :blocks] = h % (hq // hkv) == 1
            elif kind == 3:
                keep[i, h, :2] = True
            elif kind == 4:
                keep[i, h, max(blocks - 1, 0):blocks] = True
            elif kind == 5:
                keep[i, h, (h % 3):blocks:3] = True
            keep[i, h, blocks:] = rng.random(words * 32 - blocks) < 0.5
    m = np.zeros((n, hq, words), np.uint32)
    for b in range(32):
        m |= keep[:, :, b::32].astype(np.uint32) << np.uint32(b)
    c["mask"] = m.view(np.int32)


@pytest.mark.parametrize("adds,max_add", [([1] * 6, 1), ([1, 5, 1, 3, 1, 1], 5), ([20, 1, 100, 1, 40, 7], 100)])
def test_masks_that_differ_by_request_and_head(adds, max_add):
    c = attn_case(12, [9000, 300, 5000, 129, 700, 128], adds, 64, 8, 2)
    uneven_mask(c, 8, 2, 3)
    check_attn(c, run_attn(c, max_add))
    no_error()


def seen_by(c, i, pos, block_kept=None):
    """[rows of request i, heads]: does the row see the token at pos?"""
    a, b = int(c["starts"][i]), int(c["starts"][i + 1])
    hq = c["q"].shape[1]
    see = np.zeros((b - a, hq), bool)
    for t in range(b - a):
        see[t] = pos <= int(c["lens"][i]) - (b - a) + t
    if c["mask"] is not None:
        for h in range(hq):
            see[:, h] &= bool((int(c["mask"][i, h, pos // 4096]) >> (pos // 128 % 32)) & 1)
    return see


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("add", [1, 6, 90, 300])
def test_a_nan_value_reaches_the_rows_that_see_its_token_and_no_others(add, masked):
    """NaN in V early, in a block that some heads drop, among the new tokens, and at the last."""
    c = attn_case(21 + add, [1000], [add], 64, 4, 2, mask=0.6 if masked else None)
    want = run_attn(c, add)
    spots = [(3, 0, 7), (500, 1, 127), (1000 - add, 0, 64), (999, 1, 0)]
    for pos, h, dim in spots:
        c["codes"][1][c["table"][0, pos // 64], h, pos % 64, dim] = 0xFF if dim else 0x7F
    got = run_attn(c, add)
    for pos, h, dim in spots:
        see = seen_by(c, 0, pos)
        for head in (2 * h, 2 * h + 1):
            assert np.isnan(got[see[:, head], head, dim]).all(), (pos, head)
            got[see[:, head], head, dim] = want[see[:, head], head, dim]
    assert np.array_equal(got, want)
    no_error()


@pytest.mark.parametrize("add", [1, 90])
def test_a_nan_key_or_query_makes_its_rows_nan_and_no_others(add):
    c = attn_case(5, [700], [add], 32, 4, 2)
    want = run_attn(c, add)
    c["codes"][0][c["table"][0, (700 - (add + 1) // 2) // 32], 1, (700 - (add + 1) // 2) % 32, 9] = 0x7F
    c["q"][add // 2, 0, 77] = float("inf")
    c["q"][0, 1, 3] = float("nan")
    got = run_attn(c, add)
    bad = np.zeros((add, 4), bool)
    bad[:, 2:] = seen_by(c, 0, 700 - (add + 1) // 2)[:, 2:]
    bad[add // 2, 0] = bad[0, 1] = True
    assert np.isnan(got[bad]).all()
    assert np.array_equal(got[~bad], want[~bad])


def test_nothing_to_do():
    """No new tokens at all; new tokens of requests without any; one token over itself."""
    for lens, adds in (([5, 0, 300], [0, 0, 0]), ([0, 0], [0, 3]), ([1], [1])):
        for max_add in (1, 3):
            c = attn_case(1, lens, adds, 16, 4, 2, spare=3)
            check_attn(c, run_attn(c, max_add))
    no_error()


@pytest.mark.parametrize("add", [1, 70])
def test_offsets_past_32_bits(add):
    """Pages beyond 4 GB of a cache: stored, read back, attended to."""
    hkv, page, num = 8, 128, 36000
    cfg = pb.PrismCacheConfig(1, page, num, 4, 16, hkv, add, add)
    pools = [torch.empty(num, hkv, page, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.ones(num, hkv, device=DEV) for _ in range(2)]
    pages = [num - 1, 33000, 0]
    assert pages[0] * hkv * page * 128 > 2 ** 32
    g = torch.Generator().manual_seed(3)
    lens = 2 * page + 100
    whole = pb.PrismCacheConfig(1, page, num, 4, 16, hkv, lens, lens)
    slots = np.concatenate([np.arange(page) + p * page for p in pages])[:lens]
    k, v = (torch.randn(lens, hkv, 128, generator=g).bfloat16() for _ in range(2))
    pb.prism_cache_store(whole, k.to(DEV), v.to(DEV), i32(slots), *pools, *scales)
    q, o = torch.randn(add, 16, 128, generator=g).bfloat16(), torch.zeros(add, 16, 128, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(pb.prism_cache_workspace_size(cfg), dtype=torch.uint8, device=DEV)
    table = np.array([pages + [-1]], np.int32)
    pb.prism_cache_attn(cfg, q.to(DEV), *pools, *scales, i32(table), i32([lens]), i32([0, add]), o, ws)
    no_error()
    few_codes = [p[pages].cpu().numpy() for p in pools]
    few_scales = [s[pages].cpu().numpy() for s in scales]
    for x, codes, sc in zip((k, v), few_codes, few_scales):
        at = np.concatenate([np.arange(page) + i * page for i in range(3)])[:lens].astype(np.int32)
        want_c, want_s = R.store(x.double().numpy(), at, np.where(np.arange(3 * page).reshape(3, 1, page, 1) < lens, 0, codes),
                                 np.ones((3, hkv)), page)
        assert np.array_equal(codes.reshape(3, hkv, page, 128), want_c) and np.array_equal(sc, want_s)
    want, bound = R.attention(q.double().numpy(), *few_codes, *few_scales, np.array([[0, 1, 2]]), [lens], [0, add], page)
    assert (np.abs(o.double().cpu().numpy() - want) <= bound).all()


def test_prompts_in_pieces_then_tokens():
    """Two prompts of uneven pieces side by side, planned, stored and attended to piece by piece, then single tokens;
    every row against the reference on the cache as it stands."""
    hq, hkv, page, n, T = 8, 2, 16, 2, 160
    num, wide = 40, 24
    g = torch.Generator().manual_seed(8)
    ring, state = i32(np.random.default_rng(2).permutation(num)), i32([7, num, 0, 0])
    table, held, starts, slots = i32(np.full((n, wide), -1)), i32([0] * n), i32([0] * (n + 1)), i32([0] * T)
    kc, vc = (torch.full((num, hkv, page, 128), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((num, hkv), float("nan"), device=DEV) for _ in range(2))
    ws = None
    for adds in ([100, 33], [1, 60], [60, 0], [7, 8], [1, 1], [130, 1], [0, 1]):
        cfg = pb.PrismCacheConfig(n, page, num, wide, hq, hkv, T, max(adds))
        q, k, v = (torch.randn(T, h, 128, generator=g).bfloat16().to(DEV) for h in (hq, hkv, hkv))
        o = torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        pb.prism_cache_plan(cfg, held, i32(adds), ring, state, table, held, starts, slots)
        pb.prism_cache_store(cfg, k, v, slots, kc, vc, ks, vs)
        need = pb.prism_cache_workspace_size(cfg)
        if ws is None or ws.numel() < need:
            ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
        pb.prism_cache_attn(cfg, q, kc, vc, ks, vs, table, held, starts, o, ws)
        no_error()
        want, bound = R.attention(*(x.double().cpu().numpy() if x.dtype == torch.bfloat16 else x.cpu().numpy()
                                    for x in (q, kc, vc, ks, vs, table, held, starts)), page)
        live, got = ~np.isnan(want), o.double().cpu().numpy()
        assert live.sum() == sum(adds) * hq * 128 and (got[~live] == 7.0).all()
        assert (np.abs(got - want)[live] <= bound[live]).all(), adds
    assert held.tolist() == [299, 104]


def test_two_graphs_that_share_a_workspace():
    """Captured apart, replayed in turn on one stream, against the eager calls."""
    cases = [attn_case(1, [3000, 500], [1, 1], 64, 8, 2), attn_case(2, [400, 2500], [60, 3], 32, 8, 2)]
    want = [run_attn(cases[0], 1), run_attn(cases[1], 60)]
    graphs, outs, ws = [], [], None
    keep = []
    for c, add in zip(cases, (1, 60)):
        T = c["q"].shape[0]
        cfg = pb.PrismCacheConfig(2, c["page"], c["num"], c["wide"], 8, 2, T, add)
        args = (c["q"].to(DEV), *[torch.tensor(x, device=DEV) for x in c["codes"]],
                *[torch.tensor(x, device=DEV) for x in c["scales"]], i32(c["table"]), i32(c["lens"]), i32(c["starts"]))
        keep.append((cfg, args))
    ws = torch.full((max(pb.prism_cache_workspace_size(cfg) for cfg, _ in keep),), 0xFF, dtype=torch.uint8, device=DEV)
    for cfg, args in keep:
        o = torch.full(args[0].shape, 7.0, dtype=torch.bfloat16, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pb.prism_cache_attn(cfg, *args, o, ws)
        graphs.append(g)
        outs.append(o)
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert np.array_equal(w, o.double().cpu().numpy())
    no_error()


@pytest.mark.parametrize("in_place", [True, False])
def test_plan_of_many_rows_reports_a_ring_entry_that_is_no_page(in_place):
    p = Planned(6, 16, 900, 200, 9000, 3)
    p.ring[(p.state[0] + 300) % 900] = 900
    p.d["ring"] = i32(p.ring)
    assert p.step(np.array([2000, 0, 1500, 33, 2000, 1], np.int32), in_place)[4][3] == -13


def test_binding_refuses_on_the_gpu():
    c = attn_case(1, [100], [1], 16, 4, 2)
    cfg = pb.PrismCacheConfig(1, 16, c["num"], c["wide"], 4, 2, 1, 1)
    q = c["q"].to(DEV)
    pools, scales = [torch.tensor(x, device=DEV) for x in c["codes"]], [torch.tensor(x, device=DEV) for x in c["scales"]]
    ints = [i32(c["table"]), i32(c["lens"]), i32(c["starts"])]
    o, ws = torch.zeros_like(q), torch.empty(pb.prism_cache_workspace_size(cfg), dtype=torch.uint8, device=DEV)
    good = [q, *pools, *scales, *ints, o, ws]
    pb.prism_cache_attn(cfg, *good)

    def refused(at, x, kind=ValueError, **kw):
        args = list(good)
        args[at] = x
        with pytest.raises(kind):
            pb.prism_cache_attn(cfg, *args, **kw)

    refused(0, q.float())
    refused(0, q[:, :2])
    refused(0, q.cpu())
    refused(0, q.transpose(1, 2).contiguous().transpose(1, 2))
    refused(1, pools[0][:-1])
    refused(1, pools[0].transpose(1, 2))
    refused(2, pools[1].int())
    refused(3, scales[0][:1])
    refused(4, scales[1].double())
    refused(5, ints[0].long())
    refused(6, ints[1][:0])
    refused(7, ints[2][:1])
    refused(8, o.float())
    refused(8, torch.zeros(1, 8, 128, dtype=torch.bfloat16, device=DEV)[:, ::2])
    refused(9, ws[:100], pb.PrismError)
    refused(9, None, pb.PrismError)
    refused(9, "workspace")
    with pytest.raises(ValueError):
        pb.prism_cache_attn(cfg, *good, mask=i32(np.zeros((1, 3, 1))))
    no_error()


# ---------------------------------------------------------------------------
# the tile kernel by itself: calls of much work with many rows a request (a few
# such requests alone go to the few-row kernel)
# ---------------------------------------------------------------------------
def crowded(lens, adds, group, hkv):
    """The requests, and as many others of 200 new tokens as make the call much work."""
    per = -(-200 * group // 32) * (2 + 9) * hkv
    more = -(-4000 // per) + 1
    return list(lens) + [200] * more, list(adds) + [200] * more


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("lens,adds", [
    ([300, 128, 1000], [128, 128, 65]),   # whole prompts and pieces that end inside tiles
    ([257, 90, 0, 600, 1], [257, 33, 0, 90, 1]),
    ([40, 130], [50, 140]),               # rows before the first token see nothing
    ([5000], [300]),
])
def test_tiles(lens, adds, page):
    lens, adds = crowded(lens, adds, 2, 2)
    c = attn_case(sum(lens) + page, lens, adds, page, 4, 2, spare=1)
    check_attn(c, run_attn(c, max(adds)))
    no_error()


@pytest.mark.parametrize("group,add", [(1, 65), (1, 128), (1, 129), (1, 257), (3, 22), (4, 64), (5, 13), (13, 5), (13, 50),
                                       (64, 2), (64, 5)])
def test_tiles_of_every_group(group, add):
    lens, adds = crowded([add + 300, add], [add, add], group, 1)
    c = attn_case(group * 1000 + add, lens, adds, 32, group, 1, spare=2)
    check_attn(c, run_attn(c, max(adds)))
    no_error()


@pytest.mark.parametrize("mask", ["none", "first", 0.1, 0.6, "uneven"])
def test_tiles_under_masks(mask):
    lens, adds = crowded([6000, 700, 300], [150, 40, 300], 4, 2)
    c = attn_case(9, lens, adds, 64, 8, 2, mask=None if mask == "uneven" else mask)
    if mask == "uneven":
        uneven_mask(c, 8, 2, 5)
    check_attn(c, run_attn(c, max(adds)))
    no_error()


@pytest.mark.parametrize("q_layout,gap", [("heads", 0), ("fused", 0), ("packed", 4096), ("fused", 16)])
def test_tiles_of_strided_tensors(q_layout, gap):
    lens, adds = crowded([500, 77], [130, 50], 2, 3)
    c = attn_case(17, lens, adds, 16, 6, 3)
    check_attn(c, run_attn(c, max(adds), q_layout, gap))
    no_error()


@pytest.mark.parametrize("seed,kw,scale", [(1, dict(sharp=30.0), 0.0), (2, dict(sharp=0.01), 0.0), (3, dict(spread=4.0), 0.0),
                                           (4, dict(), 0.37), (5, dict(sharp=1e-30), 0.0), (6, dict(sharp=0.0), 0.0)])
def test_tiles_scales_and_sharpness(seed, kw, scale):
    lens, adds = crowded([900, 400], [70, 130], 4, 2)
    c = attn_case(seed, lens, adds, 64, 8, 2, **kw)
    check_attn(c, run_attn(c, max(adds), scale=scale), scale or None)
    no_error()


@pytest.mark.parametrize("masked", [False, True])
def test_tiles_keep_a_nan_value_to_the_rows_that_see_its_token(masked):
    lens, adds = crowded([1000], [300], 2, 2)
    c = attn_case(21, lens, adds, 64, 4, 2, mask=0.6 if masked else None)
    want = run_attn(c, 300)
    spots = [(3, 0, 7), (500, 1, 127), (700, 0, 64), (901, 1, 33), (999, 1, 0)]
    for pos, h, dim in spots:
        c["codes"][1][c["table"][0, pos // 64], h, pos % 64, dim] = 0xFF if dim else 0x7F
    got = run_attn(c, 300)
    for pos, h, dim in spots:
        see = np.zeros((len(got), 4), bool)
        see[:300] = seen_by(c, 0, pos)
        for head in (2 * h, 2 * h + 1):
            assert np.isnan(got[see[:, head], head, dim]).all(), (pos, head)
            got[see[:, head], head, dim] = want[see[:, head], head, dim]
    assert np.array_equal(got, want)
    no_error()


def test_tiles_keep_a_nan_key_or_query_to_its_rows():
    lens, adds = crowded([700], [190], 2, 2)
    c = attn_case(5, lens, adds, 32, 4, 2)
    want = run_attn(c, 200)
    c["codes"][0][c["table"][0, 600 // 32], 1, 600 % 32, 9] = 0x7F
    c["q"][95, 0, 77] = float("inf")
    c["q"][0, 1, 3] = float("nan")
    got = run_attn(c, 200)
    bad = np.zeros((len(got), 4), bool)
    bad[:190, 2:] = seen_by(c, 0, 600)[:, 2:]
    bad[95, 0] = bad[0, 1] = True
    assert np.isnan(got[bad]).all()
    assert np.array_equal(got[~bad], want[~bad])


def test_tiles_repeat_bit_for_bit_and_report_a_wrong_page():
    lens, adds = crowded([9000, 300], [100, 90], 4, 2)
    c = attn_case(6, lens, adds, 64, 8, 2)
    first = run_attn(c, 200)
    for _ in range(3):
        assert np.array_equal(first, run_attn(c, 200))
    no_error()
    c["table"][0, 2], c["table"][1, 3] = -1, c["num"]
    check_attn(c, run_attn(c, 200))
    assert pb.prism_get_last_device_error() == -13


def test_tiles_over_one_large_key_among_many():
    lens, adds = crowded([5000], [33], 4, 1)
    c = attn_case(8, lens, adds, 64, 4, 1, spread=0.0, sharp=0.2)
    page0 = c["table"][0, 0]
    q = c["q"][:33].double().numpy().mean((0, 1))
    c["q"][:33] = (0.05 * c["q"][:33].double() + torch.tensor(2.0 * np.sign(q))).bfloat16()
    c["codes"][0][page0, 0, 0] = R.encode(40.0 * np.sign(q))
    c["scales"][0][page0, 0] = 2.0 ** -5
    c["codes"][1][page0, 0, 0] = 0
    check_attn(c, run_attn(c, 200))
    no_error()


@pytest.mark.parametrize("exp", [-10, 7, 16, 23])
@pytest.mark.parametrize("lens,adds", [([300], [100]), ([40, 130], [50, 140]), ([20000], [100])])
def test_tiles_rows_that_see_nothing_beside_large_values(lens, adds, exp):
    """O is 0 for a head whose mask keeps nothing in a unit where another head's keeps all, and for rows before the
    first token, whatever the scale of V; in units of one CTA and of several (20000)."""
    n = len(lens)
    lens, adds = crowded(lens, adds, 2, 2)
    c = attn_case(40 + exp, lens, adds, 64, 4, 2, mask=0.5)
    c["scales"][1] = np.exp2(np.log2(c["scales"][1]).clip(-2, 2) + exp).astype(np.float32)
    c["mask"][:n] = -1
    c["mask"][:n, ::2] = 0
    c["mask"][n:, 0] = 0
    got = run_attn(c, max(adds))
    assert (got[:adds[0], ::2] == 0).all()
    check_attn(c, got)
    no_error()


# ---------------------------------------------------------------------------
# views
# ---------------------------------------------------------------------------
def attn_args(c, cfg, q):
    """The tensors of a call on case c, O and workspace last."""
    return [q, *[torch.tensor(x, device=DEV) for x in c["codes"]], *[torch.tensor(x, device=DEV) for x in c["scales"]],
            i32(c["table"]), i32(c["lens"]), i32(c["starts"]),
            torch.full((cfg.c.tokens, cfg.c.hq, 128), 7.0, dtype=torch.bfloat16, device=DEV),
            torch.empty(pb.prism_cache_workspace_size(cfg), dtype=torch.uint8, device=DEV)]


def test_binding_refuses_views_of_one_row():
    """O that is not of its own size, and Q, K, V of one row for all tokens and heads (strides 0, 0, which the
    library takes for packed rows)."""
    c = attn_case(3, [100, 90], [1, 2], 16, 4, 2)
    cfg = pb.PrismCacheConfig(2, 16, c["num"], c["wide"], 4, 2, 3, 2)
    good = attn_args(c, cfg, c["q"].to(DEV))
    one = torch.ones(1, 1, 128, dtype=torch.bfloat16, device=DEV)
    for at, view in ((0, one.expand(3, 4, 128)), (8, one.expand(3, 4, 128)),
                     (8, torch.zeros(1, 4, 128, dtype=torch.bfloat16, device=DEV).expand(3, 4, 128)),
                     (8, torch.zeros(3, 1, 128, dtype=torch.bfloat16, device=DEV).expand(3, 4, 128))):
        args = list(good)
        args[at] = view
        with pytest.raises(ValueError):
            pb.prism_cache_attn(cfg, *args)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device=DEV)
    for pair in ((one.expand(3, 2, 128), k), (k, one.expand(3, 2, 128))):
        with pytest.raises(ValueError):
            pb.prism_cache_store(cfg, *pair, i32([0, 1, 2]), *good[1:5])
    no_error()


@pytest.mark.parametrize("over", ["tokens", "heads", "neither"])
def test_broadcast_rows_and_dims_of_one_entry(over):
    """Q, K and V of one row for all tokens or all heads equal their copies; the stride of a dim of one entry is free."""
    hq, hkv, T = (1, 1, 5) if over == "neither" else (4, 2, 5)
    c = attn_case(3, [100, 90], [2, 3], 16, hq, hkv)
    g = torch.Generator().manual_seed(1)
    shape = {"tokens": (1, hq, 128), "heads": (T, 1, 128), "neither": (T, hq, 128)}[over]
    cfg = pb.PrismCacheConfig(2, 16, c["num"], c["wide"], hq, hkv, T, 3)
    rows = [torch.randn(shape, generator=g).bfloat16().to(DEV) for _ in range(3)]
    q, k, v = (x[:, :h].expand(T, h, 128) if over != "neither" else x.as_strided(x.shape, (128, 3, 1))
               for x, h in zip(rows, (hq, hkv, hkv)))
    slots = i32([int(c["table"][0, 0]) * 16 + x for x in range(3)] + [-1, -1])
    out = []
    for make in (lambda x: x, lambda x: x.clone(memory_format=torch.contiguous_format)):
        args = attn_args(c, cfg, make(q))
        pb.prism_cache_store(cfg, make(k), make(v), slots, *args[1:5])
        pb.prism_cache_attn(cfg, *args)
        out.append([x.view(torch.uint8) for x in args[1:9]])
    no_error()
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_one_token_of_any_stride():
    """A packed buffer of one row, whatever its stride over tokens."""
    c = attn_case(3, [100], [1], 16, 4, 2)
    cfg = pb.PrismCacheConfig(1, 16, c["num"], c["wide"], 4, 2, 1, 1)
    args = attn_args(c, cfg, c["q"].to(DEV))
    pb.prism_cache_attn(cfg, *args)
    want = args[8].clone()
    for stride in (0, 3):
        args[0], args[8] = args[0].as_strided((1, 4, 128), (stride, 128, 1)), args[8].as_strided((1, 4, 128), (stride, 128, 1))
        args[8].fill_(7.0)
        pb.prism_cache_attn(cfg, *args)
        assert torch.equal(args[8], want)
    no_error()


# ---------------------------------------------------------------------------
# small weights
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("group,add,requests", [(4, 1, 300), (4, 5, 300), (4, 70, 80)])
def test_small_weights_beside_a_sink(group, add, requests):
    """A first token that takes 0.998 of the weight and whose value is 0, before 32K tokens of 2^-24 of its weight:
    O is their sum.  Enough requests (all over the same pages) that a unit is not cut into many parts, of which one
    alone has the first token.

    The bound: a weight is fp16 times a power of two, one rounding, 2^-11 of it, or half of fp16's smallest step,
    2^-25, at a largest weight of 2^4 or more: 2^-29 of the largest (V's scales are equal).  The exponential 2^-20,
    sums in 32 bits 2^-18, dS of the score as in cache_ref.attention on both sides of the quotient, bf16 2^-8."""
    rng = np.random.default_rng(group + add)
    N, page = 32768, 64
    num = N // page
    u = rng.choice([-1.0, 1.0], 128)
    K, V = 0.25 * rng.standard_normal((N, 128)), rng.choice([-1.0, 1.0], 128) + 0.3 * rng.standard_normal((N, 128))
    K[0], V[0] = 0.75 * u, 0.0
    s = 2.0 ** -7
    codes = [R.encode(x / s) for x in (K, V)]
    K, V = (R.E4M3[x] * s for x in codes)
    Q = torch.tensor(2.0 * u + 0.02 * rng.standard_normal((add, group, 128)), dtype=torch.float32).bfloat16()
    cfg = pb.PrismCacheConfig(requests, page, num, num, group, 1, requests * add, add)
    o = torch.zeros(requests * add, group, 128, dtype=torch.bfloat16, device=DEV)
    pb.prism_cache_attn(cfg, Q.repeat(requests, 1, 1).to(DEV),
                        *[torch.tensor(x.reshape(num, 1, page, 128), device=DEV) for x in codes],
                        *[torch.full((num, 1), s, device=DEV) for _ in range(2)],
                        i32(np.tile(np.arange(num), (requests, 1))), i32([N] * requests),
                        i32(np.arange(requests + 1) * add), o,
                        torch.empty(pb.prism_cache_workspace_size(cfg), dtype=torch.uint8, device=DEV))
    no_error()
    got = o.double().cpu().numpy().reshape(requests, add, group, 128)
    q = Q.double().numpy()
    for t in range(add):
        see = N - add + t + 1
        for h in range(group):
            score = K[:see] @ q[t, h] / np.sqrt(128.0)
            p = np.exp(score - score.max())
            p /= p.sum()
            dS = (2.0 ** -17 * np.abs(q[t, h]).max() * np.abs(K).sum(1).max() +
                  2.0 ** -20 * (np.abs(K) @ np.abs(q[t, h])).max()) / np.sqrt(128.0)
            want, pv = p @ V[:see], p @ np.abs(V[:see])
            bound = 2.0 ** -8 * np.abs(want) + 1.01 * (2.0 ** -11 + 2.0 ** -18 + 2.0 ** -20 + 2 * dS) * pv + \
                1.01 * 2.0 ** -29 * p.max() * np.abs(V[:see] / s).sum(0) * s
            assert p[0] > 0.997 and (bound < 0.1 * np.abs(want)).all()  # (a lost part would be seen)
            assert (np.abs(got[:, t, h] - want) <= bound).all(), (t, h, np.abs(got[:, t, h] / want - 1).max())


# ---------------------------------------------------------------------------
# what is reported
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("add", [1, 6, 200])
def test_dropped_blocks_need_no_page(add, page):
    """Table entries of blocks that every head drops may be anything, beside kept ones too; one that a kept block
    reads is reported."""
    lens, adds = ([9000], [add]) if add < 200 else crowded([9000], [add], 2, 2)
    c = attn_case(3, lens, adds, page, 4, 2, mask=1.0)
    dropped = [b for b in range(71) if b % 5]  # of 71 blocks
    for b in dropped:
        c["mask"][0, :, b // 32] &= ~np.int32(np.uint32(1 << (b % 32)).view(np.int32))
        c["table"][0, b * 128 // page:-(-min((b + 1) * 128, 9000) // page)] = (-1, c["num"])[b % 2]
    got = run_attn(c, max(adds))
    no_error()
    check_attn(c, got)
    c["table"][0, 10 * 128 // page] = -1  # (block 10 is kept)
    check_attn(c, run_attn(c, max(adds)))
    assert pb.prism_get_last_device_error() == -13


@pytest.mark.parametrize("max_add", [1, 70])
@pytest.mark.parametrize("what", ["len<0", "len>room", "start<0", "starts descend", "starts past the rows"])
def test_lengths_and_offsets_outside_are_clamped_and_reported(what, max_add):
    c = attn_case(4, [300, 200, 90], [max_add, 1, 3], 32, 4, 2, spare=2)
    lens, starts = c["lens"].copy(), c["starts"].copy()
    if what == "len<0":
        c["lens"][1], lens[1] = -7, 0
    elif what == "len>room":  # every entry of the row is read
        c["table"][0] = c["table"][0, 0]
        c["lens"][0], lens[0] = c["wide"] * 32 + 1, c["wide"] * 32
        for codes in c["codes"]:
            codes[codes == 0x7F] = 0x38
    elif what == "start<0":
        c["starts"][0], starts[0] = -2 ** 31, 0
    elif what == "starts descend":  # the last request has no rows
        c["starts"][3], starts[3] = max_add, max_add + 1
    else:
        c["starts"][3], starts[3] = 2 ** 31 - 1, len(c["q"])
    got = run_attn(c, max_add)
    assert pb.prism_get_last_device_error() == -13
    check_attn(dict(c, lens=lens, starts=starts), got)
    c["lens"], c["starts"] = lens, starts
    run_attn(c, max_add)
    no_error()


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("tokens", [200, 9000])  # one CTA, several
def test_plan_reports_a_returned_entry_that_is_no_page(tokens, in_place):
    p = Planned(3, 16, 40, 9, tokens, 5)
    p.step(np.array([50, 20, 0], np.int32), in_place)
    no_error()
    p.table[0, 2] = 40
    p.d["table"] = i32(p.table)
    add, d = np.array([-1, 1, 5], np.int32), p.d
    want = R.plan(p.held, add, p.ring, p.state, p.table, 16, tokens)
    lens, out = (d["held"], d["state"]) if in_place else (d["lens"], i32([5, 5, 0, 5]))
    pb.prism_cache_plan(p.cfg, d["held"], i32(add), d["ring"], d["state"], d["table"], lens, d["starts"], d["slots"], out)
    assert pb.prism_get_last_device_error() == -13
    for w, g in zip(want, (lens, d["starts"], d["slots"], d["ring"], out, d["table"])):
        assert np.array_equal(w, g.cpu().numpy())
    assert want[4][3] == 0 and 40 in want[3]


def test_binding_refuses_rows_of_another_length():
    """A table, mask or scales with enough entries in rows that are not the config's (they would be read askew)."""
    c = attn_case(3, [100, 90], [1, 2], 16, 4, 2, mask=0.5)
    cfg = pb.PrismCacheConfig(2, 16, c["num"], c["wide"], 4, 2, 3, 2)
    good, mask = attn_args(c, cfg, c["q"].to(DEV)), i32(c["mask"])
    pb.prism_cache_attn(cfg, *good, mask=mask)
    pb.prism_cache_attn(cfg, *good[:5], good[5].view(-1), *good[6:], mask=mask.view(-1))
    pb.prism_cache_attn(cfg, *good[:5], torch.cat([good[5]] * 2), *good[6:], mask=mask.view(8, -1))
    wide = torch.cat([good[5]] * 2, 1)
    for at, x in ((5, wide), (3, good[3].t().contiguous()), (4, good[4].view(1, -1))):
        args = list(good)
        args[at] = x
        with pytest.raises(ValueError):
            pb.prism_cache_attn(cfg, *args)
    for m in (torch.cat([mask] * 2, 2), torch.cat([mask] * 2, 1), torch.cat([mask.view(8, -1)] * 2, 1)):
        with pytest.raises(ValueError):
            pb.prism_cache_attn(cfg, *good, mask=m)
    n = [i32([0] * 4) for _ in range(4)]
    with pytest.raises(ValueError):
        pb.prism_cache_plan(cfg, n[0], n[1], i32([0] * c["num"]), n[2], wide, n[0], n[3], i32([0] * 3))
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        pb.prism_cache_store(cfg, k, k, i32([0, 1, 2]), good[1], good[2], good[3].t().contiguous(), good[4])
    no_error()


# ---------------------------------------------------------------------------
# the tile kernel's own offsets, counters and parts
# ---------------------------------------------------------------------------
def rule_constants():
    """The sizes that choose between the kernels, from the sources."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(pb.__file__), "csrc")
    text = "".join(open(os.path.join(csrc, f)).read() for f in ("cache_attention.cuh", "prism.cu"))
    return {k: int(re.search(rf"\b{k} = (\d+)", text).group(1))
            for k in ("kLittleWork", "kFewUnitRows", "kFewUnitCost", "kCacheFewRows")}


def takes_tiles(lens, adds, group, hkv, max_add):
    """Does a call run the tile kernel?  (As its comment says: places of the requests of many rows.)"""
    k = rule_constants()
    if max_add * group <= k["kCacheFewRows"]:
        return False
    many = [(-(-a * group // k["kFewUnitRows"])) * (max(-(-n // 128), 1) + k["kFewUnitCost"]) * hkv
            for n, a in zip(lens, adds) if a * group > k["kCacheFewRows"]]
    return sum(many) > k["kLittleWork"]


@pytest.mark.parametrize("nan", [False, True])
def test_tiles_offsets_past_32_bits(nan):
    """Pages beyond 4 GB of a cache, read by TMA and, for a NaN among their values, directly."""
    hkv, hq, page, num, add, n = 8, 16, 128, 36000, 200, 4
    held = 2 * page + 100
    assert takes_tiles([held] * n, [add] * n, hq // hkv, hkv, add)
    pools = [torch.empty(num, hkv, page, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.ones(num, hkv, device=DEV) for _ in range(2)]
    pages = [num - 1, 33000, 0]
    assert pages[1] * hkv * page * 128 > 2 ** 32
    g = torch.Generator().manual_seed(4)
    slots = np.concatenate([np.arange(page) + p * page for p in pages])[:held]
    k, v = (torch.randn(held, hkv, 128, generator=g).bfloat16() for _ in range(2))
    if nan:
        v[130, 3, 77] = float("nan")
    pb.prism_cache_store(pb.PrismCacheConfig(1, page, num, 4, hq, hkv, held, held), k.to(DEV), v.to(DEV), i32(slots),
                         *pools, *scales)
    cfg = pb.PrismCacheConfig(n, page, num, 4, hq, hkv, n * add, add)
    q = torch.randn(n * add, hq, 128, generator=g).bfloat16()
    o = torch.zeros(n * add, hq, 128, dtype=torch.bfloat16, device=DEV)
    starts = np.arange(n + 1) * add
    pb.prism_cache_attn(cfg, q.to(DEV), *pools, *scales, i32([pages + [-1]] * n), i32([held] * n), i32(starts), o,
                        torch.empty(pb.prism_cache_workspace_size(cfg), dtype=torch.uint8, device=DEV))
    no_error()
    codes, got = [x[pages].cpu().numpy() for x in pools], o.double().cpu().numpy()
    if nan:
        assert (codes[1][1, 3, 2, 77] & 0x7F) == 0x7F
        codes[1][1, 3, 2, 77] = 0
    want, bound = R.attention(q.double().numpy(), *codes, *[x[pages].cpu().numpy() for x in scales],
                              np.array([[0, 1, 2]] * n), [held] * n, starts, page)
    if nan:  # every row of heads 6 and 7 sees token 130 (the first new one is 156)
        assert np.isnan(got[:, 6:8, 77]).all()
        want[:, 6:8, 77] = got[:, 6:8, 77] = 0
    assert (np.abs(got - want) <= bound).all()


def test_tiles_of_prompts_in_pieces():
    """Eight prompts side by side, planned, stored and attended to piece by piece, single tokens between."""
    hq, hkv, page, n, T = 8, 2, 32, 8, 1700
    num, wide = 200, 24
    g = torch.Generator().manual_seed(9)
    ring, state = i32(np.random.default_rng(2).permutation(num)), i32([7, num, 0, 0])
    table, held, starts, slots = i32(np.full((n, wide), -1)), i32([0] * n), i32([0] * (n + 1)), i32([0] * T)
    kc, vc = (torch.full((num, hkv, page, 128), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((num, hkv), float("nan"), device=DEV) for _ in range(2))
    cfg = pb.PrismCacheConfig(n, page, num, wide, hq, hkv, T, 220)
    ws = torch.full((pb.prism_cache_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device=DEV)
    for adds, tiles in (([200, 220, 180, 210, 199, 201, 220, 220], True), ([1, 1, 0, 3, 1, 1, 1, 1], False),
                        ([190, 200, 1, 210, 180, 201, 220, 220], True), ([1] * 8, False)):
        q, k, v = (torch.randn(T, h, 128, generator=g).bfloat16().to(DEV) for h in (hq, hkv, hkv))
        o = torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        pb.prism_cache_plan(cfg, held, i32(adds), ring, state, table, held, starts, slots)
        pb.prism_cache_store(cfg, k, v, slots, kc, vc, ks, vs)
        pb.prism_cache_attn(cfg, q, kc, vc, ks, vs, table, held, starts, o, ws)
        no_error()
        assert takes_tiles(held.tolist(), adds, hq // hkv, hkv, 220) == tiles
        want, bound = R.attention(*(x.double().cpu().numpy() if x.dtype == torch.bfloat16 else x.cpu().numpy()
                                    for x in (q, kc, vc, ks, vs, table, held, starts)), page)
        live, got = ~np.isnan(want), o.double().cpu().numpy()
        assert live.sum() == sum(adds) * hq * 128 and (got[~live] == 7.0).all()
        assert (np.abs(got - want)[live] <= bound[live]).all(), adds


def test_replays_that_move_between_the_kernels_and_share_a_workspace():
    """Two graphs on one workspace, replayed in turn with lengths that send their requests to the tile kernel, to the
    few-row kernel and back; each replay equals the eager call."""
    group, hkv, page, n, most = 4, 2, 64, 6, 230
    sizes = [([900, 5000, 700, 230, 400, 1200], [230, 90, 200, 230, 17, 220], True),
             ([901, 5001, 90, 1, 400, 1200], [1, 90, 3, 1, 17, 1], False),
             ([20, 8000, 300, 300, 300, 999], [20, 200, 220, 230, 1, 200], True)]
    for lens, adds, tiles in sizes:
        assert takes_tiles(lens, adds, group, hkv, most) == tiles
    T = max(sum(a) for _, a, _ in sizes)
    graphs, cfgs = [], []
    cases = [[attn_case(10 * j + i, lens, adds, page, group * hkv, hkv, spare=T - sum(adds))
              for i, (lens, adds, _) in enumerate(sizes)] for j in range(2)]
    num, wide = (max(c[k] for cs in cases for c in cs) for k in ("num", "wide"))
    for cs in cases:
        for c in cs:  # one cache and table size for all
            c["codes"] = [np.concatenate([x, np.zeros((num - c["num"],) + x.shape[1:], np.uint8)]) for x in c["codes"]]
            c["scales"] = [np.concatenate([x, np.ones((num - c["num"], hkv), np.float32)]) for x in c["scales"]]
            c["table"] = np.pad(c["table"], ((0, 0), (0, wide - c["wide"])), constant_values=-1)
            c["num"], c["wide"] = num, wide
    cfg = pb.PrismCacheConfig(n, page, num, wide, group * hkv, hkv, T, most)
    bufs = [attn_args(cs[0], cfg, cs[0]["q"].to(DEV)) for cs in cases]
    bufs[1][9] = bufs[0][9].fill_(0xFF)
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pb.prism_cache_attn(cfg, *b)
        graphs.append(g)
    want = [[run_attn(c, most) for c in cs] for cs in cases]
    check_attn(cases[0][0], want[0][0])
    check_attn(cases[1][1], want[1][1])
    for turn in range(9):
        at = [turn % 3, (turn // 3 + turn) % 3]
        for b, cs, i in zip(bufs, cases, at):
            for x, y in zip(b, (cs[i]["q"], *cs[i]["codes"], *cs[i]["scales"], cs[i]["table"], cs[i]["lens"], cs[i]["starts"])):
                x.copy_(torch.as_tensor(y))
            b[8].fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b, w, i in zip(bufs, want, at):
            assert np.array_equal(b[8].double().cpu().numpy(), w[i])
    no_error()


@pytest.mark.parametrize("size", [8, 11, 14, 17])
@pytest.mark.parametrize("add", [1, 6, 200])
def test_scores_far_beyond_the_exponentials_range(add, size):
    """Scores up to 2^(2 size + 4): where the largest leads by more than its own rounding, O is that token's V (one
    weight of 1: fp16's rounding 2^-11, bf16's 2^-8, the quotient's).  The last places of such scores are larger than
    the exponents that P can hold."""
    lens, adds = ([700, 30, 3], [add, 1, 3]) if add < 200 else crowded([700, 230], [add, 230], 2, 2)
    assert takes_tiles(lens, adds, 2, 2, max(adds)) == (add == 200)
    c = attn_case(size, lens, adds, 64, 4, 2, spread=0.0, sharp=1.0)
    c["q"] = (c["q"].double() * 2.0 ** size).bfloat16()
    c["scales"][0] = (c["scales"][0] * 2.0 ** size).astype(np.float32)
    got, q = run_attn(c, max(adds)), c["q"].double().numpy()
    no_error()
    assert np.isfinite(got).all()
    checked = rows = 0
    for i, total in enumerate(c["lens"]):
        a, b = int(c["starts"][i]), int(c["starts"][i + 1])
        pos = np.arange(total)
        pg = c["table"][i][pos // 64]
        for h in range(4):
            K, V = (R.E4M3[x[pg, h // 2, pos % 64]] * s[pg, h // 2][:, None].astype(np.float64)
                    for x, s in zip(c["codes"], c["scales"]))
            score = q[a:b, h] @ K.T / np.sqrt(128.0)
            score[pos[None] > total - (b - a) + np.arange(b - a)[:, None]] = -np.inf
            err = (2.0 ** -17 * np.abs(q[a:b, h]).max(1) * np.abs(K).sum(1).max() +
                   2.0 ** -20 * (np.abs(q[a:b, h]) @ np.abs(K).T).max(1)) / np.sqrt(128.0)
            best = score.argmax(1)
            lead = score[np.arange(b - a), best] - np.partition(score, -2, 1)[:, -2] if total > 1 else np.full(b - a, np.inf)
            sure = lead > 2 * err + 40  # (the others' weights are below e^-40)
            rows, checked = rows + len(sure), checked + sure.sum()
            assert (np.abs(got[a:b, h] - V[best]) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(V[best]))[sure].all(), (i, h)
    assert checked > 0.8 * rows


@pytest.mark.parametrize("what", ["len<0", "start<0", "starts past the rows"])
def test_lengths_and_offsets_outside_are_reported_under_a_mask(what):
    c = attn_case(4, [300, 200, 90], [1, 1, 1], 32, 4, 2, mask=0.7, spare=2)
    lens, starts = c["lens"].copy(), c["starts"].copy()
    if what == "len<0":
        c["lens"][1], lens[1] = -7, 0
    elif what == "start<0":
        c["starts"][0], starts[0] = -5, 0
    else:
        c["starts"][3], starts[3] = 99, len(c["q"])
    got = run_attn(c, 1)
    assert pb.prism_get_last_device_error() == -13
    check_attn(dict(c, lens=lens, starts=starts), got)
    c["lens"], c["starts"] = lens, starts
    run_attn(c, 1)
    no_error()
