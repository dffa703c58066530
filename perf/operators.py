"""Cases of the paged 8-bit cache: its plan, its store and the attention over it.

Three operators, in the order in which a serving program calls them for each
step:

  plan    block tables, packed row offsets and slot numbers from the request
          lengths, pages handed out from (and returned to) a ring of free pages;
  store   keys and values of new tokens into e4m3 pages, one power-of-two scale
          for each page and KV head;
  attn    causal attention of the new tokens over their requests' pages, with an
          optional block mask for each request and query head.

With ``own`` false, ``run`` computes them from elementary torch operations in 32
bits; with ``own`` true it calls the library.  ``exact`` is each operator's
definition in 64 bits, request by request.

A step's lengths come from the case alone (``mix`` seeds them), the tensors from
the seed.
"""
import math
import random

import torch

own = False

D = 128          # head dim
BLOCK = 128      # tokens a mask bit stands for
MIN_EXP = -64    # the smallest page scale is 2^-64
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a serving batch: most requests stay in their last page
        {"name": "plan_step", "op": "plan", "requests": 64, "page": 64, "lo": 1, "hi": 8192, "add_lo": 1, "add_hi": 1,
         "ended": 0, "spare": 0, "mix": 1},
        # prompts that arrive together while other requests end and return their pages
        {"name": "plan_prompts", "op": "plan", "requests": 1000, "page": 16, "lo": 0, "hi": 2000, "add_lo": 0,
         "add_hi": 500, "ended": 5, "spare": 77, "mix": 2},
        # the new token of each request of a decode batch
        {"name": "store_step", "op": "store", "requests": 64, "page": 64, "hkv": 8, "lo": 1, "hi": 8192, "add_lo": 1,
         "add_hi": 1, "heads_first": False, "spare": 0, "mix": 3},
        # ragged pieces of prompts that begin and end inside pages, and a padded tail
        {"name": "store_pieces", "op": "store", "requests": 7, "page": 32, "hkv": 5, "lo": 0, "hi": 999, "add_lo": 1,
         "add_hi": 1500, "heads_first": False, "spare": 41, "mix": 4},
        # one whole prompt as a prefill layer holds it, heads first
        {"name": "store_prompt", "op": "store", "requests": 1, "page": 128, "hkv": 8, "lo": 0, "hi": 0,
         "add_lo": 131072, "add_hi": 131072, "heads_first": True, "spare": 0, "mix": 5},
        # the smallest call: one chat turn's next token
        {"name": "attn_single", "op": "attn", "requests": 1, "page": 16, "hq": 32, "hkv": 8, "lo": 777, "hi": 777,
         "add_lo": 1, "add_hi": 1, "density": 1.0, "spare": 0, "mix": 6},
        # a decode batch of mixed ages
        {"name": "attn_step", "op": "attn", "requests": 64, "page": 64, "hq": 32, "hkv": 8, "lo": 1, "hi": 16384,
         "add_lo": 1, "add_hi": 1, "density": 1.0, "spare": 0, "mix": 7},
        # one token after the longest prompt of the benchmark
        {"name": "attn_long", "op": "attn", "requests": 1, "page": 128, "hq": 32, "hkv": 8, "lo": 131072, "hi": 131072,
         "add_lo": 1, "add_hi": 1, "density": 1.0, "spare": 0, "mix": 8},
        # several long prompts: the largest read of the cache
        {"name": "attn_long_batch", "op": "attn", "requests": 6, "page": 128, "hq": 32, "hkv": 8, "lo": 60001,
         "hi": 131072, "add_lo": 1, "add_hi": 1, "density": 1.0, "spare": 0, "mix": 9},
        # long prompts under a block mask as the estimator makes them
        {"name": "attn_masked", "op": "attn", "requests": 8, "page": 64, "hq": 32, "hkv": 8, "lo": 30000, "hi": 131000,
         "add_lo": 1, "add_hi": 1, "density": 0.18, "spare": 0, "mix": 10},
        # five drafted tokens a request to verify, and padded rows
        {"name": "attn_draft", "op": "attn", "requests": 32, "page": 32, "hq": 32, "hkv": 8, "lo": 100, "hi": 8191,
         "add_lo": 5, "add_hi": 5, "density": 1.0, "spare": 11, "mix": 11},
        # the next piece of two long prompts
        {"name": "attn_piece", "op": "attn", "requests": 2, "page": 64, "hq": 32, "hkv": 8, "lo": 20000, "hi": 32768,
         "add_lo": 1800, "add_hi": 2048, "density": 1.0, "spare": 0, "mix": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "attn", "attn", "attn"])
    c = {"op": op, "page": rng.choice([16, 32, 64, 128]), "spare": rng.choice([0, 0, rng.randint(1, 99)]),
         "mix": rng.randint(100, 10 ** 6)}
    if op == "plan":
        c["requests"] = _log_int(rng, 1, 1000)
        c["lo"], c["hi"] = 0, _log_int(rng, 1, 2000)
        c["add_hi"] = 1 if rng.random() < 0.5 else _log_int(rng, 2, 500)
        c["add_lo"] = rng.choice([0, 1])
        c["ended"] = rng.choice([0, 5])
    elif op == "store":
        c["requests"] = 1 if rng.random() < 0.3 else _log_int(rng, 2, 200)
        c["hkv"] = rng.choice([1, 2, 5, 8])
        c["lo"], c["hi"] = 0, _log_int(rng, 1, 5000)
        c["add_lo"], c["add_hi"] = 1, 1 if rng.random() < 0.4 else _log_int(rng, 2, 80000 // c["requests"])
        c["heads_first"] = rng.random() < 0.4
    else:
        c["hq"], c["hkv"] = rng.choice([(32, 8), (32, 8), (1, 1), (8, 8), (12, 2), (20, 4), (64, 8)])
        kind = rng.choice(["step", "step", "draft", "piece"])
        c["requests"] = _log_int(rng, 1, 4 if kind == "piece" else 100)
        # the cache read stays under the largest listed one, the products under the largest piece
        most = min(131072, 500000 * 8 // (c["requests"] * c["hkv"]), 40000 if kind == "piece" else 131072)
        c["hi"] = _log_int(rng, 1, most)
        c["lo"] = rng.randint(0, c["hi"])
        if kind == "step":
            c["add_lo"] = c["add_hi"] = 1
        elif kind == "draft":
            c["add_lo"], c["add_hi"] = 1, rng.randint(2, 8)
        else:
            c["add_lo"], c["add_hi"] = 1, _log_int(rng, 16, 2000 // c["requests"])
        c["density"] = rng.choice([1.0, 1.0, round(rng.uniform(0.1, 0.9), 2)])
    return c


def _lengths(c):
    """(held, add) of every request: the tokens it has and those that it brings (-1: it ends)."""
    r = random.Random(c["mix"])
    held = [r.randint(c["lo"], c["hi"]) for _ in range(c["requests"])]
    add = [r.randint(c["add_lo"], c["add_hi"]) for _ in range(c["requests"])]
    if c.get("ended"):
        add = [-1 if i % c["ended"] == 2 else a for i, a in enumerate(add)]
    return held, add


def _pages(n, page):
    return -(-n // page)


def _blocks(c, total):
    """Ranks of the kept blocks of a masked request: how many a KV head keeps, always the last block among them."""
    nblk = _pages(total, BLOCK)
    return max(1, round(c["density"] * nblk))


def work(c):
    held, add = _lengths(c)
    new = [max(a, 0) for a in add]
    if c["op"] == "plan":
        opened = sum(_pages(h + a, c["page"]) - _pages(h, c["page"]) for h, a in zip(held, new))
        freed = sum(_pages(h, c["page"]) for h, a in zip(held, add) if a < 0)
        part = sum(1 for h, a in zip(held, new) if a and h % c["page"])
        # held, add, lens, starts; slots; ring and table of opened and returned pages; tables of begun pages; the state
        moved = 4 * (4 * len(held) + 1) + 4 * (sum(new) + c["spare"]) + 8 * (opened + freed) + 4 * part + 24
        return {"bytes": moved, "flops": 0}
    if c["op"] == "store":
        rows = sum(new) * c["hkv"]
        touched = sum(_pages(h + a, c["page"]) - h // c["page"] for h, a in zip(held, new)) * c["hkv"]
        return {"bytes": rows * D * (4 + 2) + 8 * touched + 4 * (sum(new) + c["spare"]), "flops": 0}
    g, kv, pairs, pages = c["hq"] // c["hkv"], 0, 0, 0
    for h, a in zip(held, new):
        total = h + a
        if c["density"] >= 1.0:
            kv += total
            pairs += c["hq"] * sum(range(h + 1, total + 1))
            pages += _pages(total, c["page"])
        else:
            kb, last = _blocks(c, total), total - (_pages(total, BLOCK) - 1) * BLOCK
            kv += (kb - 1) * BLOCK + last
            dropped = [sum(1 for rank in range(kb - 1) if g > 1 and rank % g == j) for j in range(g)]
            pairs += c["hkv"] * a * sum((kb - 1 - d) * BLOCK + last for d in dropped)
            pages += kb * max(1, BLOCK // c["page"])
    rows = sum(new) * c["hq"]
    return {"bytes": kv * c["hkv"] * 2 * D + pages * (8 * c["hkv"] + 4) + rows * D * 4, "flops": 4 * D * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cells(c, gen, need, extra):
    """Pages of the requests in random order: (num_pages, max_pages, table with -1 behind each request's pages, the free pages)."""
    num = sum(need) + extra
    order = torch.randperm(num, generator=gen, device=DEV).to(torch.int32)
    wide = max(need) + 3
    n = torch.tensor(need, device=DEV)
    first = torch.cumsum(n, 0) - n
    col = torch.arange(wide, device=DEV)
    at = (first[:, None] + col).clamp(max=num - 1)
    table = torch.where(col < n[:, None], order[at], torch.full_like(order[at], -1))
    return num, wide, table, order[sum(need):]


def _page_scale(amax):
    """The smallest power of two s >= 2^MIN_EXP with amax / s <= 448 = 1.75 * 2^8 (amax in fp32, >= 0)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return ((e + 127) << 23).view(torch.float32)


def _filled(gen, num, hkv, page):
    """Codes and scales of a cache whose pages hold keys or values of varying size."""
    mean = torch.randn(1, hkv, 1, D, generator=gen, device=DEV)
    size = torch.exp(0.7 * torch.randn(num, hkv, 1, 1, generator=gen, device=DEV))
    x = torch.randn(num, hkv, page, D, generator=gen, device=DEV).mul_(0.5).add_(mean).mul_(size)
    s = _page_scale(x.abs().amax((2, 3)))
    return x.div_(s[:, :, None, None]).to(torch.float8_e4m3fn), s, mean


def _slots(held, add, table, page, spare):
    """Slots of the new tokens, packed request after request, then `spare` rows of -1."""
    h, a = torch.tensor(held, device=DEV), torch.tensor(add, device=DEV)
    total = int(sum(add))
    i = torch.repeat_interleave(torch.arange(len(add), device=DEV), a, output_size=total)
    pos = h[i] + torch.arange(total, device=DEV) - (torch.cumsum(a, 0) - a)[i]
    s = table[i, pos // page].long() * page + pos % page
    return torch.cat([s, torch.full((spare,), -1, device=DEV)]).to(torch.int32)


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    held, add = _lengths(c)
    new = [max(a, 0) for a in add]
    page, n, tokens = c["page"], c["requests"], max(1, sum(new) + c["spare"])
    st = {"op": c["op"], "page": page}
    have = [_pages(h, page) for h in held]
    need = [_pages(h + a, page) for h, a in zip(held, new)]
    if c["op"] == "plan":
        opened = sum(need) - sum(have)
        num, _, table, free = _cells(c, gen, have, opened + 5 + n // 4)
        wide = max(need) + 3
        table = torch.nn.functional.pad(table[:, :wide], (0, max(0, wide - table.shape[1])), value=-1).contiguous()
        head = int(torch.randint(0, num, (1,), generator=gen, device=DEV))
        ring = torch.full((num,), -1, dtype=torch.int32, device=DEV)
        ring[(head + torch.arange(free.numel(), device=DEV)) % num] = free
        st.update(held=_i32(held), add=_i32(add), ring=ring, state=_i32([head, free.numel(), 0, 0]), table=table,
                  lens=_i32([0] * n), starts=_i32([0] * (n + 1)), slots=_i32([0] * tokens), state_out=_i32([0] * 4))
        hq = hkv = 1
    elif c["op"] == "store":
        hq = hkv = c["hkv"]
        num, wide, table, _ = _cells(c, gen, [t - h // page for t, h in zip(need, held)], 3)
        slots = _slots([h % page for h in held], new, table, page, tokens - sum(new))
        kc, ks, _ = _filled(gen, num, hkv, page)
        vc, vs, _ = _filled(gen, num, hkv, page)
        shape = (hkv, tokens, D) if c["heads_first"] else (tokens, hkv, D)
        k = (2 * torch.randn(shape, generator=gen, device=DEV)).bfloat16()
        v = torch.randn(shape, generator=gen, device=DEV).bfloat16()
        if c["heads_first"]:
            k, v = k.transpose(0, 1), v.transpose(0, 1)
        st.update(k=k, v=v, slots=slots, kc=kc, vc=vc, ks=ks, vs=vs)
    else:
        hq, hkv = c["hq"], c["hkv"]
        num, wide, table, _ = _cells(c, gen, need, 2)
        kc, ks, mean = _filled(gen, num, hkv, page)
        vc, vs, _ = _filled(gen, num, hkv, page)
        lens = [h + a for h, a in zip(held, new)]
        # cells behind a request's last token were never written: NaN codes
        col = torch.arange(page, device=DEV)
        last = torch.stack([table[i, m - 1] for i, m in enumerate(need)]).long()
        tail = col >= (_i32(lens) - (_i32(need) - 1) * page)[:, None]
        for x in (kc.view(torch.uint8), vc.view(torch.uint8)):
            x[last] = torch.where(tail[:, None, :, None], torch.full_like(x[last], 0x7f), x[last])
        q = 2 * torch.randn(tokens, hkv, hq // hkv, D, generator=gen, device=DEV) + mean.view(1, hkv, 1, D)
        mask = None
        if c["density"] < 1.0:
            words = _pages(wide * page, 32 * BLOCK)
            keep = torch.zeros(n, hkv, hq // hkv, words * 32, dtype=torch.bool, device=DEV)
            for i, total in enumerate(lens):
                nblk, kb = _pages(total, BLOCK), _blocks(c, total)
                pick = torch.rand(hkv, nblk - 1, generator=gen, device=DEV).argsort(1)[:, :kb - 1].sort(1).values
                rank = torch.arange(kb - 1, device=DEV)
                for j in range(hq // hkv):
                    mine = pick[:, rank % (hq // hkv) != j] if hq > hkv else pick
                    keep[i, :, j].scatter_(1, mine, True)
                keep[i, :, :, nblk - 1] = True
            bits = keep.view(n, hq, words, 32).long() << torch.arange(32, device=DEV)
            mask = bits.sum(-1)
            mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(torch.int32)
        starts = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
        starts[1:] = torch.cumsum(_i32(new), 0)
        st.update(q=q.reshape(tokens, hq, D).bfloat16(), kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=_i32(lens),
                  starts=starts, mask=mask, o=torch.randn(tokens, hq, D, generator=gen, device=DEV).bfloat16(),
                  max_len=max(lens), max_add=max(new))
    if own:
        import block_sparse_attention_band_b200 as pb
        cfg = pb.PrismCacheConfig(n, page, num, wide, hq, hkv, tokens, max(1, max(new)))
        st["cfg"] = cfg
        if c["op"] == "attn":
            st["ws"] = torch.empty(pb.prism_cache_workspace_size(cfg), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    if own:
        return {"plan": _own_plan, "store": _own_store, "attn": _own_attn}[st["op"]](st)
    return {"plan": _plain_plan, "store": _plain_store, "attn": _plain_attn}[st["op"]](st)


def _own_plan(st):
    import block_sparse_attention_band_b200 as pb
    pb.prism_cache_plan(st["cfg"], st["held"], st["add"], st["ring"], st["state"], st["table"], st["lens"],
                        st["starts"], st["slots"], st["state_out"])
    return {k: st[k] for k in ("table", "lens", "starts", "slots", "ring", "state_out")}


def _own_store(st):
    import block_sparse_attention_band_b200 as pb
    pb.prism_cache_store(st["cfg"], st["k"], st["v"], st["slots"], st["kc"], st["vc"], st["ks"], st["vs"])
    return {k: st[k] for k in ("kc", "vc", "ks", "vs")}


def _own_attn(st):
    import block_sparse_attention_band_b200 as pb
    pb.prism_cache_attn(st["cfg"], st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"], st["lens"],
                        st["starts"], st["o"], st["ws"], mask=st["mask"])
    return st["o"]


def _plain_plan(st):
    page, num, tokens = st["page"], st["ring"].numel(), st["slots"].numel()
    held, add, table, ring = st["held"].long(), st["add"].long(), st["table"], st["ring"]
    n, wide = table.shape
    new, have = add.clamp(min=0), (held + page - 1) // page
    need = (held + new + page - 1) // page - have
    back = torch.where(add < 0, have, torch.zeros_like(have))
    ends, need_to, back_to = torch.cumsum(new, 0), torch.cumsum(need, 0), torch.cumsum(back, 0)
    head, count = st["state"][0].long(), st["state"][1].long()
    # new tokens: the request of each, its position, its page
    t = torch.arange(tokens, device=held.device)
    i = torch.searchsorted(ends, t, right=True).clamp(max=n - 1)
    real = t < ends[-1]
    pos = held[i] + t - (ends - new)[i]
    j = (pos // page).clamp(0, wide - 1)
    fresh = ring[(head + (need_to - need)[i] + j - have[i]) % num].long()
    pg = torch.where(j >= have[i], fresh, table[i, j].long())
    slots = torch.where(real, pg * page + pos % page, torch.full_like(pos, -1))
    # opened pages into the table, pages of ended requests behind the ring's last (one cell more takes what is not written)
    opens = real & (j >= have[i]) & (pos % page == 0)
    cells = torch.cat([table.reshape(-1), table.new_zeros(1)])
    cells[torch.where(opens, i * wide + j, torch.full_like(i, n * wide))] = pg.to(torch.int32)
    col = torch.arange(wide, device=held.device)
    at = (head + count + (back_to - back)[:, None] + col) % num
    rings = torch.cat([ring, ring.new_zeros(1)])
    rings[torch.where(col < back[:, None], at, torch.full_like(at, num))] = table
    zero = torch.zeros_like(head)
    state = torch.stack([(head + need_to[-1]) % num, count - need_to[-1] + back_to[-1], zero, zero])
    lens = torch.where(add < 0, torch.zeros_like(held), held + new)
    starts = torch.cat([zero[None], ends])
    return {"table": cells[:-1].view(n, wide), "lens": lens.int(), "starts": starts.int(), "slots": slots.int(),
            "ring": rings[:-1], "state_out": state.int()}


def _plain_store(st):
    page, slots = st["page"], st["slots"].long()
    num, hkv = st["ks"].shape
    real = slots >= 0
    pg = torch.where(real, slots // page, torch.full_like(slots, num))
    off = torch.where(real, slots % page, torch.full_like(slots, page))
    first = torch.full((num + 1,), page, device=slots.device).scatter_reduce(0, pg, off, "amin")[:num]
    cell = torch.where(real, pg * page + off, torch.full_like(slots, num * page))
    for x, codes, scales in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
        x = x.float()
        top = torch.zeros(num + 1, hkv, device=x.device)
        top = top.scatter_reduce(0, pg[:, None].expand(-1, hkv), x.abs().amax(2), "amax")[:num]
        # a page written from its first cell forgets its old scale
        scale = torch.maximum(_page_scale(top), torch.where((first == 0)[:, None], torch.zeros_like(scales), scales))
        scale = torch.where((first < page)[:, None], scale, scales)
        # older codes of a page that was begun before, at the new scale
        older = torch.nonzero((first > 0) & (first < page))[:, 0]
        was = codes[older].float()
        at = (was * (scales / scale)[older][:, :, None, None]).to(codes.dtype).float()
        keep = torch.arange(page, device=x.device) >= first[older][:, None]
        codes.view(torch.uint8)[older] = torch.where(keep[:, None, :, None], was, at).to(codes.dtype).view(torch.uint8)
        scales.copy_(scale)
        q = (x / scale[pg.clamp(max=num - 1)][:, :, None]).to(codes.dtype).view(torch.uint8)
        flat = codes.view(torch.uint8)
        live = torch.nonzero(real)[:, 0]
        flat[pg[live], :, off[live]] = q[live]
    return {k: st[k] for k in ("kc", "vc", "ks", "vs")}


def _plain_attn(st):
    page, table, lens, starts = st["page"], st["table"], st["lens"].long(), st["starts"].long()
    tokens, hq, _ = st["q"].shape
    num, hkv = st["ks"].shape
    n, g, wide, long = table.shape[0], hq // hkv, st["max_add"], st["max_len"]
    dev = table.device
    pages = table[:, :_pages(long, page)].long().clamp(0, num - 1)
    pos = torch.arange(pages.shape[1] * page, device=dev)
    held = (pos < lens[:, None])[:, None, :, None]

    def values(codes, scales):
        x = codes[pages].float() * scales[pages][..., None, None]      # [n, pages, hkv, page, D]
        x = x.transpose(1, 2).reshape(n, hkv, -1, D)
        return torch.where(held, x, torch.zeros_like(x))

    qlen = starts[1:] - starts[:-1]
    t = torch.arange(wide, device=dev)
    row = starts[:-1, None] + t
    q = st["q"][row.clamp(max=tokens - 1)].float().view(n, wide, hkv, g, D)
    q = q.permute(0, 2, 3, 1, 4).reshape(n, hkv, g * wide, D)
    s = (q @ values(st["kc"], st["ks"]).transpose(2, 3)) * (1.0 / math.sqrt(D))
    s = s.view(n, hkv, g, wide, -1)
    seen = (pos <= (lens - qlen)[:, None, None] + t[:, None])[:, None, None]
    if st["mask"] is not None:
        word = st["mask"].view(n, hkv, g, -1)[..., pos // (32 * BLOCK)].long()
        seen = seen & (((word >> (pos // BLOCK % 32)) & 1) == 1)[:, :, :, None]
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    o = (p.view(n, hkv, g * wide, -1) @ values(st["vc"], st["vs"])).view(n, hkv, g, wide, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(n * wide, hq, D).bfloat16()
    # rows of no request stay as they were
    out = torch.cat([st["o"], st["o"][:1]])
    out[torch.where(t < qlen[:, None], row, torch.full_like(row, tokens)).view(-1)] = o
    return out[:-1]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    if c["op"] == "plan":
        return None  # whole numbers
    st = prepare(c, seed)
    page = c["page"]
    if c["op"] == "store":
        slots = st["slots"].cpu().tolist()
        runs, at = [], 0
        while at < len(slots) and slots[at] >= 0:
            end = at + 1
            while end < len(slots) and slots[end] >= 0 and slots[end] // page == slots[at] // page:
                end += 1
            runs.append((slots[at] // page, slots[at] % page, at, end))
            at = end
        out = {}
        for x, codes, scales in (("k", "kc", "ks"), ("v", "vc", "vs")):
            src, value, scale = st[x].double(), st[codes].double(), st[scales].double()
            for pg, off, a, b in runs:
                new = src[a:b].transpose(0, 1)                       # [hkv, tokens, D]
                top = new.abs().amax((1, 2))
                # a power of two below the scale, doubled until 448 of it reach the largest value
                s = _power_of_two(torch.log2(top / 448).floor().clamp(min=MIN_EXP + 1) - 1)
                for _ in range(3):
                    s = torch.where(448 * s < top, 2 * s, s)
                if off:
                    s = torch.maximum(s, scale[pg])
                    back = value[pg, :, :off] * (scale[pg] / s)[:, None, None]
                    value[pg, :, :off] = _to_e4m3(back)
                scale[pg] = s
                value[pg, :, off:off + b - a] = _to_e4m3(new / s[:, None, None])
            out[codes], out[scales] = value, scale
        return out
    hq, hkv = c["hq"], c["hkv"]
    g = hq // hkv
    out = st["o"].double()
    starts, lens = st["starts"].tolist(), st["lens"].tolist()
    for i, total in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        pages = st["table"][i, :_pages(total, page)].long()
        limit = torch.arange(total - (b - a), total, device=DEV)
        pos = torch.arange(total, device=DEV)
        for h in range(hkv):
            k, v = ((st[x][pages, h].double() * st[y][pages, h].double()[:, None, None]).reshape(-1, D)[:total]
                    for x, y in (("kc", "ks"), ("vc", "vs")))
            for j in range(h * g, h * g + g):
                s = st["q"][a:b, j].double() @ k.T / math.sqrt(D)
                see = pos[None] <= limit[:, None]
                if st["mask"] is not None:
                    w = st["mask"][i, j].long() & 0xffffffff
                    see = see & ((w[pos // 4096] >> (pos // 128 % 32)) & 1).bool()[None]
                s[~see] = -math.inf
                out[a:b, j] = torch.softmax(s, 1).nan_to_num(0.0) @ v
    return out


def _power_of_two(e):
    """2^e in 64 bits, from its bits (a power function rounds)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _to_e4m3(x):
    """The nearest e4m3 value (ties to even) of a 64-bit x with |x| <= 448: 3 bits behind the leading one, steps of 2^-9 at least."""
    _, e = torch.frexp(x)
    step = _power_of_two((e - 4).clamp(min=-9))
    return torch.round(x / step) * step
