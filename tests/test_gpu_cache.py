"""The paged 8-bit cache on the GPU against the 64-bit reference (cache_ref):
plan and store bit for bit, the attention within the bound derived there."""
import numpy as np
import pytest
import torch

import block_sparse_attention_band_b200 as pb
from tests import cache_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def no_error():
    torch.cuda.synchronize()
    assert pb.prism_get_last_device_error() == 0


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------
class Planned:
    """Device buffers of a plan and the reference's copy."""

    def __init__(self, n, page, num, wide, tokens, seed):
        rng = np.random.default_rng(seed)
        self.page, self.tokens = page, tokens
        self.ring, self.state = rng.permutation(num).astype(np.int32), np.array([int(rng.integers(num)), num, 0, 0])
        self.table, self.held = np.full((n, wide), -7, np.int32), np.zeros(n, np.int32)
        self.cfg = pb.PrismCacheConfig(n, page, num, wide, 1, 1, tokens, 1)
        self.d = {"held": i32(self.held), "ring": i32(self.ring), "state": i32(self.state), "table": i32(self.table),
                  "lens": i32(self.held * 0 - 9), "starts": i32(np.full(n + 1, -9)), "slots": i32(np.full(tokens, -9))}

    def step(self, add, in_place):
        d = self.d
        out = d["state"] if in_place else i32([5, 5, 0, 5])
        lens = d["held"] if in_place else d["lens"]
        pb.prism_cache_plan(self.cfg, d["held"], i32(add), d["ring"], d["state"], d["table"], lens, d["starts"],
                            d["slots"], out)
        torch.cuda.synchronize()
        want = R.plan(self.held, add, self.ring, self.state, self.table, self.page, self.tokens)
        got = (lens, d["starts"], d["slots"], d["ring"], out, d["table"])
        for name, w, g in zip(("lens", "starts", "slots", "ring", "state", "table"), want, got):
            assert np.array_equal(w, g.cpu().numpy()), name
        self.held, _, _, self.ring, self.state, self.table = want
        assert pb.prism_get_last_device_error() == self.state[3]
        if not in_place:
            d["held"], d["state"] = lens.clone(), out.clone()
        return want


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("n,page,num,wide,tokens,most", [
    (1, 16, 9, 8, 130, 60), (5, 32, 40, 9, 300, 70), (70, 128, 300, 5, 5000, 100), (300, 16, 3000, 11, 6000, 33),
    (4096, 64, 9000, 3, 40000, 9),
])
def test_plan_steps_match(n, page, num, wide, tokens, most, in_place):
    """Requests that grow, idle and end over several steps, some of which do not fit."""
    p = Planned(n, page, num, wide, tokens, n + page)
    rng = np.random.default_rng(n)
    failed = 0
    for step in range(12):
        add = np.where(rng.random(n) < 0.15, -1, rng.integers(0, most, n)).astype(np.int32)
        failed += p.step(add, in_place)[4][3] != 0
    assert failed < 12


def test_plan_one_long_prompt_and_padding():
    p = Planned(1, 16, 9000, 8500, 140000, 4)
    p.step(np.array([131072 + 5], np.int32), True)
    p.step(np.array([1], np.int32), True)
    p.step(np.array([-1], np.int32), True)


@pytest.mark.parametrize("why", ["rows", "pages", "length", "held<0", "held>room", "add<-1", "begun", "begun<0", "state",
                                 "count"])
@pytest.mark.parametrize("tokens", [40, 5000])  # one CTA, several
def test_plan_step_that_does_not_fit_changes_nothing(why, tokens):
    p = Planned(4, 16, 12, 8, tokens, 1)
    p.step(np.array([5, 9, 0, 16], np.int32), True)
    add = np.array([1, 1, 1, 1], np.int32)
    if why == "rows":
        p.cfg.c.tokens = p.tokens = 3
        p.d["slots"] = p.d["slots"][:3].contiguous()
    elif why == "pages":
        add[:] = [40, 40, 40, 40] if tokens == 5000 else [10, 10, 10, 10]
        if tokens == 40:
            p.state[1] = 1
    elif why == "length":
        add[1] = 16 * 8
        p.cfg.c.tokens = p.tokens = max(tokens, 200)
        p.d["slots"] = i32(np.zeros(p.tokens))
    elif why == "held<0":
        p.held[2] = -1
    elif why == "held>room":
        p.held[0] = 16 * 8 + 1
    elif why == "add<-1":
        add[3] = -2
    elif why == "begun":
        p.table[0, 0] = 12
    elif why == "begun<0":
        p.table[1, 0] = -1
    elif why == "state":
        p.state[0] = 12
    elif why == "count":
        p.state[1] = 13
    for k in ("held", "table", "state"):
        p.d[k] = i32(getattr(p, k))
    assert p.step(add, True)[4][3] == -13


def test_plan_ring_entry_that_is_no_page():
    p = Planned(3, 16, 10, 4, 60, 2)
    p.ring[(p.state[0] + 1) % 10] = 10
    p.ring[(p.state[0] + 2) % 10] = -4
    p.d["ring"] = i32(p.ring)
    assert p.step(np.array([17, 3, 16], np.int32), True)[4][3] == -13


# ---------------------------------------------------------------------------
# store
# ---------------------------------------------------------------------------
def store_case(seed, page, hkv, runs, tail, spread=0.0):
    """Runs (place in the page at which it begins, rows) packed one after the other, -1 rows between and behind them."""
    rng = np.random.default_rng(seed)
    num = sum(-(-(o + n) // page) for o, n in runs) + 2
    order = rng.permutation(num)
    slots, at = [], 0
    for o, n in runs:
        for pos in range(o, o + n):
            slots.append(order[at + pos // page] * page + pos % page)
        at += -(-(o + n) // page)
        slots += [-1] * int(rng.integers(0, 2))
    slots = np.array(slots + [-1] * tail, np.int32)
    codes = rng.integers(0, 256, (2, num, hkv, page, 128)).astype(np.uint8)
    codes[(codes & 127) == 127] = 0x38
    scales = 2.0 ** rng.integers(-10, -6, (2, num, hkv))
    x = rng.standard_normal((2, len(slots), hkv, 128)) * np.exp(spread * rng.standard_normal((2, len(slots), hkv, 1)))
    x = torch.tensor(x, dtype=torch.float32).bfloat16()
    return slots, codes, scales.astype(np.float32), x


def check_store(slots, codes, scales, x, page, max_add, layout="packed", gap=0):
    T, hkv = x.shape[1:3]
    num = codes.shape[1]
    dense = hkv * page * 128
    cfg = pb.PrismCacheConfig(1, page, num, num, hkv, hkv, T, max_add, page_stride=dense + gap if gap else 0)
    if layout == "packed":
        k, v = x[0].to(DEV), x[1].to(DEV)
    elif layout == "heads":
        k, v = (y.transpose(0, 1).contiguous().to(DEV).transpose(0, 1) for y in x)
    else:  # slices of one fused projection
        both = torch.zeros(T, 3 * hkv, 128, dtype=torch.bfloat16, device=DEV)
        both[:, hkv:2 * hkv], both[:, 2 * hkv:] = x[0].to(DEV), x[1].to(DEV)
        k, v = both[:, hkv:2 * hkv], both[:, 2 * hkv:]
    pools = []
    for c in codes:
        pool = torch.full((num, dense + gap), 0x55, dtype=torch.uint8, device=DEV)
        pool[:, :dense] = torch.tensor(c.reshape(num, -1), device=DEV)
        pools.append(pool)
    views = [p[:, :dense].view(num, hkv, page, 128) for p in pools]
    ds = [torch.tensor(s, device=DEV) for s in scales]
    pb.prism_cache_store(cfg, k, v, i32(slots), views[0], views[1], ds[0], ds[1])
    no_error()
    for which in range(2):
        want_c, want_s = R.store(x[which].double().numpy(), slots, codes[which], scales[which], page)
        assert np.array_equal(ds[which].double().cpu().numpy(), want_s)
        got = views[which].cpu().numpy()
        same = (got == want_c) | (((got & 127) == 127) & ((want_c & 127) == 127))  # (a NaN has two codes)
        assert same.all(), (which, np.argwhere(~same)[:5])
        assert (pools[which][:, dense:] == 0x55).all()


@pytest.mark.parametrize("layout", ["packed", "heads", "fused"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_store_ragged_runs(page, layout):
    runs = [(0, 1), (page - 1, 1), (5, page), (0, 3 * page + 7), (page // 2, 1), (3, 2), (0, page), (page - 1, 2)]
    case = store_case(page, page, 3, runs, 5, spread=1.0)
    check_store(*case, page, 3 * page + 7, layout)


@pytest.mark.parametrize("max_add", [1, 2, 7, 40, 1000])
@pytest.mark.parametrize("page", [16, 128])
def test_store_result_does_not_depend_on_max_add(page, max_add):
    runs = [(i % page, 1 + i % 5) for i in range(0, 60, 3)] + [(0, 700), (9, 250)]
    case = store_case(7, page, 2, runs, 40, spread=0.5)
    check_store(*case, page, max_add)


@pytest.mark.parametrize("page", [16, 64])
def test_store_scale_growth_and_extremes(page):
    """Begun pages whose scale grows by much or little or not at all; zeros; the range's ends; odd values."""
    runs = [(page - 3, 2)] * 9 + [(0, 2)] * 9
    slots, codes, scales, x = store_case(3, page, 1, runs, 0)
    amps = [2.0 ** 30, 2.0 ** -30, 0.0, 3.0, 3e38, 2.0 ** -80, 2.0 ** -130, 447.9, 1.0]
    starts = np.flatnonzero((slots >= 0) & (np.concatenate([[-1], slots[:-1]]) // page != slots // page))
    for i, t in enumerate(starts):
        x[:, t:t + 2] = (torch.tanh(x[:, t:t + 2].double()) * amps[i % 9]).bfloat16()
    check_store(slots, codes, scales, x, page, 2)


def test_store_nan_and_infinity():
    slots, codes, scales, x = store_case(5, 32, 2, [(0, 40), (7, 3), (31, 1), (2, 1)], 2)
    x[0, 3, 0, 5], x[0, 4, 1, 77], x[1, 9, 0, 0] = float("nan"), float("inf"), float("-inf")
    t = int(np.flatnonzero(slots >= 0)[-1])
    x[:, t] = float("inf")  # a row of nothing finite in a begun page
    x[0, t, 0] = float("nan")
    check_store(slots, codes, scales, x, 32, 40)


def test_store_pages_apart():
    slots, codes, scales, x = store_case(11, 64, 2, [(0, 130), (63, 4), (1, 1)], 3)
    check_store(slots, codes, scales, x, 64, 130, gap=2 * 64 * 128 + 4096)


def test_store_slot_outside_the_cache_is_skipped_and_reported():
    slots, codes, scales, x = store_case(2, 16, 1, [(0, 20)], 3)
    num = codes.shape[1]
    wrong = slots.copy()
    wrong[-3:] = [num * 16, 2 ** 31 - 1, -5]
    pools = [torch.tensor(c, device=DEV) for c in codes]
    ds = [torch.tensor(s, device=DEV) for s in scales]
    cfg = pb.PrismCacheConfig(1, 16, num, num, 1, 1, len(slots), 20)
    pb.prism_cache_store(cfg, x[0].to(DEV), x[1].to(DEV), i32(wrong), *pools, *ds)
    torch.cuda.synchronize()
    assert pb.prism_get_last_device_error() == -13
    for which in range(2):
        want_c, want_s = R.store(x[which].double().numpy(), slots, codes[which], scales[which], 16)
        assert np.array_equal(pools[which].cpu().numpy(), want_c) and np.array_equal(ds[which].cpu().numpy(), want_s)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attn_case(seed, lens, adds, page, hq, hkv, mask=None, spare=0, spread=0.7, sharp=2.0, q_scale=1.0):
    rng = np.random.default_rng(seed)
    n = len(lens)
    need = [-(-max(x, 0) // page) for x in lens]
    num = sum(need) + 3
    order = rng.permutation(num)
    wide = max(need + [1]) + 2
    table = rng.integers(-5, num + 5, (n, wide)).astype(np.int32)  # (behind the last page: anything)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    codes, scales = [], []
    for _ in range(2):
        mean = rng.standard_normal((1, hkv, 1, 128))
        x = (mean + 0.5 * rng.standard_normal((num, hkv, page, 128))) * np.exp(
            spread * rng.standard_normal((num, hkv, 1, 1)))
        s = 2.0 ** np.ceil(np.log2(np.abs(x).max((2, 3)) / 448))
        codes.append(R.encode(x / s[:, :, None, None]))
        scales.append(s.astype(np.float32))
    for i, x in enumerate(lens):  # places behind the last token: NaN codes
        if x > 0 and x % page:
            for c in codes:
                c[table[i, need[i] - 1], :, x % page:] = 0x7F
    starts = np.concatenate([[0], np.cumsum(adds)]).astype(np.int32)
    T = max(1, int(starts[-1]) + spare)
    q = torch.tensor(sharp * q_scale * rng.standard_normal((T, hq, 128)), dtype=torch.float32).bfloat16()
    words = (-(-wide * page // 128) + 31) // 32
    m = None
    if mask is not None:
        blocks = words * 32
        if mask == "none":
            keep = np.zeros((n, hq, blocks), bool)
        elif mask == "first":
            keep = np.zeros((n, hq, blocks), bool)
            keep[:, ::2, 0] = True
        else:
            keep = rng.random((n, hq, blocks)) < mask
        m = np.zeros((n, hq, words), np.uint32)
        for b in range(32):
            m |= keep[:, :, b::32].astype(np.uint32) << np.uint32(b)
        m = m.view(np.int32)
    return dict(q=q, codes=codes, scales=scales, table=table, lens=np.array(lens, np.int32), starts=starts, mask=m,
                page=page, num=num, wide=wide)


def run_attn(c, max_add, q_layout="packed", gap=0, scale=0.0, ws=None):
    T, hq, _ = c["q"].shape
    num, hkv, page = c["num"], c["scales"][0].shape[1], c["page"]
    dense = hkv * page * 128
    cfg = pb.PrismCacheConfig(len(c["lens"]), page, num, c["wide"], hq, hkv, T, max_add, softmax_scale=scale,
                              page_stride=dense + gap if gap else 0)
    q = c["q"].to(DEV)
    if q_layout == "heads":
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    elif q_layout == "fused":
        both = torch.full((T, hq + 2 * hkv, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
        both[:, :hq] = q
        q = both[:, :hq]
    pools = []
    for x in c["codes"]:
        pool = torch.full((num, dense + gap), 0x7F, dtype=torch.uint8, device=DEV)
        pool[:, :dense] = torch.tensor(x.reshape(num, -1), device=DEV)
        pools.append(pool[:, :dense].view(num, hkv, page, 128))
    if ws is None:
        ws = torch.full((pb.prism_cache_workspace_size(cfg),), 0xFF, dtype=torch.uint8, device=DEV)
    o = torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    pb.prism_cache_attn(cfg, q, *pools, *[torch.tensor(s, device=DEV) for s in c["scales"]], i32(c["table"]),
                        i32(c["lens"]), i32(c["starts"]), o, ws, mask=None if c["mask"] is None else i32(c["mask"]))
    torch.cuda.synchronize()
    return o.double().cpu().numpy()


def check_attn(c, got, scale=None):
    want, bound = R.attention(c["q"].double().numpy(), *c["codes"], *c["scales"], c["table"], c["lens"], c["starts"],
                              c["page"], c["mask"], scale)
    live = ~np.isnan(want)
    assert (got[~live] == 7.0).all(), "rows of no request were written"
    over = np.abs(got[live] - want[live]) - bound[live]
    assert np.isfinite(got[live]).all()
    assert (over <= 0).all(), (over.max(), np.argwhere(np.abs(np.where(live, got - want, 0)) > np.where(live, bound, 1))[:5])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (5, 1), (32, 8)])
def test_attn_single_tokens(hq, hkv, page):
    lens = [1, 2, page - 1, page, page + 1, 127, 128, 129, 300, 1000, 777]
    c = attn_case(page + hq, lens, [1] * len(lens), page, hq, hkv, spare=3)
    check_attn(c, run_attn(c, 1))
    no_error()


@pytest.mark.parametrize("group", [2, 3, 7, 16, 17, 33, 64])
def test_attn_group_sizes(group):
    lens, adds = [200, 1, 513], [1, 1, 3]
    c = attn_case(group, lens, adds, 64, 2 * group, 2)
    check_attn(c, run_attn(c, 3))
    no_error()


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("lens,adds,max_add", [
    ([5, 300, 128, 1000], [5, 2, 128, 7], 128),             # whole prompts among drafts
    ([700, 129], [257, 129], 257),                          # pieces that end inside tiles
    ([90, 40, 0, 600, 1], [3, 0, 0, 9, 1], 9),              # requests without rows, without tokens
    ([3, 0, 130], [5, 2, 140], 140),                        # rows before the first token see nothing
    ([2000], [1000], 1),                                    # more rows than expected
    ([260, 260], [1, 1], 2),
])
def test_attn_several_rows(lens, adds, max_add, page):
    c = attn_case(sum(lens) + page, lens, adds, page, 4, 2, spare=1)
    check_attn(c, run_attn(c, max_add))
    no_error()


@pytest.mark.parametrize("mask", ["none", "first", 0.1, 0.5, 0.95])
@pytest.mark.parametrize("adds,max_add", [([1, 1, 1], 1), ([1, 4, 2], 4), ([1, 150, 40], 150)])
def test_attn_masks(mask, adds, max_add):
    c = attn_case(len(adds) + max_add, [1500, 700, 6000], adds, 32, 8, 2, mask=mask)
    check_attn(c, run_attn(c, max_add))
    no_error()


@pytest.mark.parametrize("q_layout,gap", [("heads", 0), ("fused", 0), ("packed", 4096), ("fused", 16)])
@pytest.mark.parametrize("max_add", [1, 60])
def test_attn_layouts(q_layout, gap, max_add):
    adds = [1, 1, 1] if max_add == 1 else [1, 60, 5]
    c = attn_case(17, [100, 500, 77], adds, 16, 6, 3)
    check_attn(c, run_attn(c, max_add, q_layout, gap))
    no_error()


@pytest.mark.parametrize("max_add", [1, 70])
def test_attn_scales_and_sharpness(max_add):
    """Sharp and flat softmax, pages of very different size, a softmax scale of its own, tiny and zero queries."""
    adds = [1, 1] if max_add == 1 else [70, 3]
    for seed, kw, scale in ((1, dict(sharp=30.0), 0.0), (2, dict(sharp=0.01), 0.0), (3, dict(spread=4.0), 0.0),
                            (4, dict(), 0.37), (5, dict(sharp=1e-30), 0.0), (6, dict(sharp=0.0), 0.0)):
        c = attn_case(seed, [900, 400], adds, 64, 8, 2, **kw)
        check_attn(c, run_attn(c, max_add, scale=scale), scale or None)
    no_error()


@pytest.mark.parametrize("max_add", [1, 33])
def test_attn_one_large_key_among_many(max_add):
    """A first token that takes most of the weight and whose value is zero: what is left is the small weights' sum."""
    adds = [max_add]
    c = attn_case(8, [5000], adds, 64, 2, 1, spread=0.0, sharp=0.2)
    page0 = c["table"][0, 0]
    q = c["q"].double().numpy().mean((0, 1))
    c["q"] = (0.05 * c["q"].double() + torch.tensor(2.0 * np.sign(q))).bfloat16()
    c["codes"][0][page0, 0, 0] = R.encode(40.0 * np.sign(q) / 1.0)
    c["scales"][0][page0, 0] = 2.0 ** -5
    c["codes"][1][page0, 0, 0] = 0
    check_attn(c, run_attn(c, max_add))
    no_error()


@pytest.mark.parametrize("hq,hkv,page", [(8, 2, 64), (4, 1, 16)])
def test_attn_long(hq, hkv, page):
    c = attn_case(31, [70001, 33, 40000], [1, 1, 1], page, hq, hkv)
    check_attn(c, run_attn(c, 1))
    no_error()


def test_attn_many_requests():
    rng = np.random.default_rng(0)
    lens = rng.integers(1, 400, 300).tolist()
    c = attn_case(77, lens, [1] * 300, 32, 4, 2)
    check_attn(c, run_attn(c, 1))
    no_error()


@pytest.mark.parametrize("max_add", [1, 40])
def test_attn_table_entry_that_is_no_page_is_left_out_and_reported(max_add):
    c = attn_case(5, [300, 200], [max_add, 1], 32, 4, 2)
    c["table"][0, 2], c["table"][0, 5], c["table"][1, 0] = -1, c["num"], 2 ** 31 - 1
    check_attn(c, run_attn(c, max_add))
    assert pb.prism_get_last_device_error() == -13


@pytest.mark.parametrize("max_add", [1, 50])
def test_attn_repeats_bit_for_bit_and_leaves_the_workspace_free(max_add):
    c = attn_case(6, [9000, 50, 3000], [max_add, 1, 1], 64, 8, 2)
    first = run_attn(c, max_add)
    for _ in range(3):
        assert np.array_equal(first, run_attn(c, max_add))


def test_attn_nan_values_reach_only_the_rows_that_see_them():
    c = attn_case(9, [200, 200], [1, 1], 64, 4, 2)
    want = run_attn(c, 1)
    c["codes"][1][c["table"][0, 1], 0, 3, 7] = 0x7F
    got = run_attn(c, 1)
    assert np.isnan(got[0, :2, 7]).all()
    got[0, :2, 7] = want[0, :2, 7]
    assert np.array_equal(got, want)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_prefill_then_decode_in_a_replayed_graph():
    """A prompt through prism_prefill, its K and V into the cache, then decode steps replayed from one graph, masked
    by the estimator's last row; each step's O against the reference on the cache as it stands."""
    from tests import gen
    hq, hkv, N, page, n = 4, 2, 640, 64, 3
    hi, lo = gen.default_bands()
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(1, h, N, 128, generator=g).bfloat16().to(DEV) for h in (hq, hkv, hkv))
    cfg = pb.PrismConfig(1, hq, hkv, N, hi, lo, 0.6)
    ws = torch.empty(pb.prism_workspace_size(cfg), dtype=torch.uint8, device=DEV)
    mask = torch.empty(1, hq, cfg.nb, cfg.words, dtype=torch.int32, device=DEV)
    pb.prism_prefill(cfg, q, k, v, mask, torch.empty_like(q), ws)

    num, wide = 40, 12
    ring, state = i32(np.random.default_rng(1).permutation(num)), i32([3, num, 0, 0])
    table, held, starts = i32(np.full((n, wide), -1)), i32([0] * n), i32([0] * (n + 1))
    kc, vc = (torch.full((num, hkv, page, 128), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((num, hkv), float("nan"), device=DEV) for _ in range(2))
    # request 1 is the prompt, the others begin empty
    whole = pb.PrismCacheConfig(n, page, num, wide, hq, hkv, N, N)
    slots = i32([0] * N)
    pb.prism_cache_plan(whole, held, i32([0, N, 0]), ring, state, table, held, starts, slots)
    pb.prism_cache_store(whole, k[0].transpose(0, 1), v[0].transpose(0, 1), slots, kc, vc, ks, vs)
    no_error()

    step = pb.PrismCacheConfig(n, page, num, wide, hq, hkv, 4, 1)
    words = step.words
    keep = torch.full((n, hq, words), -1, dtype=torch.int32, device=DEV)
    keep[1, :, 0] = mask[0, :, -1, 0] | (-1 << cfg.nb)  # new blocks are kept
    qs, knew, vnew = (torch.zeros(4, h, 128, dtype=torch.bfloat16, device=DEV) for h in (hq, hkv, hkv))
    o = torch.full((4, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    add, slots = i32([1, 1, 0]), i32([0] * 4)
    aws = torch.empty(pb.prism_cache_workspace_size(step), dtype=torch.uint8, device=DEV)

    def one():
        pb.prism_cache_plan(step, held, add, ring, state, table, held, starts, slots)
        pb.prism_cache_store(step, knew, vnew, slots, kc, vc, ks, vs)
        pb.prism_cache_attn(step, qs, kc, vc, ks, vs, table, held, starts, o, aws, mask=keep)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    sizes = []
    for it in range(70):
        for x in (qs, knew, vnew):
            x.copy_(torch.randn(x.shape, generator=g).bfloat16() * (1 + it % 3))
        add.copy_(i32([1, 1, 1 if it > 40 else 0]) if it != 60 else i32([-1, 1, 1]))
        graph.replay()
        torch.cuda.synchronize()
        sizes.append(held.tolist())
        if it in (0, 1, 39, 41, 60, 63, 69):
            got = o.double().cpu().numpy()
            want, bound = R.attention(qs.double().cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), ks.cpu().numpy(),
                                      vs.cpu().numpy(), table.cpu().numpy(), held.cpu().numpy(), starts.cpu().numpy(),
                                      page, keep.cpu().numpy())
            live = ~np.isnan(want)
            assert (np.abs(got - want)[live] <= bound[live]).all(), it
    no_error()
    assert sizes[0] == [1, 641, 0] and sizes[59] == [60, 700, 19] and sizes[69] == [9, 710, 29]
    assert state.tolist()[1] + sum(-(-x // page) for x in sizes[-1]) == num and state.tolist()[2:] == [0, 0]


def test_steps_on_two_streams_with_two_workspaces():
    c = [attn_case(s, [3000, 800], [1, 1], 64, 8, 2) for s in (1, 2)]
    want = [run_attn(x, 1) for x in c]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    prepared, outs = [], []
    for x in c:
        cfg = pb.PrismCacheConfig(2, 64, x["num"], x["wide"], 8, 2, 2, 1)
        prepared.append((cfg, x["q"].to(DEV), *[torch.tensor(y, device=DEV) for y in x["codes"]],
                         *[torch.tensor(y, device=DEV) for y in x["scales"]], i32(x["table"]), i32(x["lens"]),
                         i32(x["starts"])))
        outs.append((torch.empty(2, 8, 128, dtype=torch.bfloat16, device=DEV),
                     torch.empty(pb.prism_cache_workspace_size(cfg), dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, a, b in zip(streams, prepared, outs):
            with torch.cuda.stream(s):
                pb.prism_cache_attn(*a, *b)
    torch.cuda.synchronize()
    for w, (o, _) in zip(want, outs):
        assert np.array_equal(w, o.double().cpu().numpy())
