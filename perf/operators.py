"""Cases, plain forms and 64-bit values of the paged-cache operators.

Three operators serve a paged, dictionary-coded KV cache.  A page holds
``page`` token slots of every KV head; a slot is one key record and one value
record of 16 code words (fp16 coefficient << 16 | atom index), so the pool is
int32 [n_pages][Hkv][page][2][16].

* tables: block tables, slot maps and row offsets of a step from the
  requests' lengths, pages taken from a stack of free ones;
* store:  code words of new tokens written to their slots;
* attend: attention of every request's new tokens over its paged codes,
  K_t = sum_j c_tj D_K[i_tj], V_t = sum_j c_tj D_V[i_tj],
  out_i = sum_t softmax_t(scale <q_i, K_t>) V_t, t up to the token's own
  position (and within the window where there is one).

``run`` computes them with elementary torch operations, or, where ``own`` is
set, with the package's entry points.
"""

import math
import random

import torch

own = False

K_ATOMS = 16


# ------------------------------------------------------------------- cases

def listed():
    full = dict(Hq=32, Hkv=8, d=128, atoms=32768)
    return [
        # one generated token for four long requests: the smallest plan of a serving step
        dict(name="tables_step_b4", op="tables", B=4, page=64, max_len=32768, max_new=1, shape=0),
        # one generated token for each of 256 requests of mixed lengths
        dict(name="tables_step_b256", op="tables", B=256, page=16, max_len=32768, max_new=1, shape=7),
        # prompts of up to 16384 tokens entering together, lengths of every kind
        dict(name="tables_prompts_b64", op="tables", B=64, page=64, max_len=32768, max_new=16384,
             shape=11),
        # the codes of one generated token for each of four requests
        dict(name="store_step_b4", op="store", T=4, Hkv=8, page=64),
        # the codes of a 16384-token prompt
        dict(name="store_prompt_16k", op="store", T=16384, Hkv=8, page=64),
        # one token for each of eight short chats: latency is all
        dict(name="step_short_b8", op="attend", B=8, max_len=600, max_new=1, window=0, page=16,
             shape=3, **full),
        # the 32K, batch-4 generation step
        dict(name="step_32k_b4", op="attend", B=4, max_len=32768, max_new=1, window=0, page=64,
             shape=0, **full),
        # one token over the longest context served
        dict(name="step_256k", op="attend", B=1, max_len=262144, max_new=1, window=0, page=128,
             shape=0, **full),
        # a few drafted tokens of each of eight requests checked at once
        dict(name="draft_4k_b8", op="attend", B=8, max_len=4096, max_new=5, window=0, page=64,
             shape=5, **full),
        # a whole 4096-token prompt, nothing before it
        dict(name="prompt_4k", op="attend", B=1, max_len=4096, max_new=4096, window=0, page=64,
             shape=0, **full),
        # a 2048-token piece of a long prompt, 30720 tokens behind it
        dict(name="chunk_2k_of_32k", op="attend", B=1, max_len=32768, max_new=2048, window=0,
             page=64, shape=0, **full),
        # pieces and single tokens of twelve requests in one call, 64-dim heads, a window, odd pages
        dict(name="mixed_window_d64", op="attend", B=12, max_len=5001, max_new=701, window=1024,
             page=24, shape=17, Hq=4, Hkv=1, d=64, atoms=1024),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "store", "attend", "attend", "attend"])
    if op == "tables":
        B = _log(rng, 1, 512)
        return dict(op=op, B=B, page=rng.choice([8, 16, 24, 64, 100, 128]),
                    max_len=_log(rng, 64, 65536),
                    max_new=_log(rng, 1, max(1, min(16384, 1048576 // B))),
                    shape=rng.randrange(1, 1 << 30))
    if op == "store":
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, T=_log(rng, 1, 131072 // Hkv), Hkv=Hkv, page=rng.choice([8, 16, 24, 64, 128]))
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 8]) if Hkv < 8 else rng.choice([1, 2, 3, 4])
    max_new = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 2048)])
    # scored pairs and rebuilt vectors stay below those of the largest listed cases
    B = _log(rng, 1, 16)
    hi = min(262144 * 8 // (Hkv * B), 1000000000 // (B * Hkv * g * max_new), 262144)
    max_len = _log(rng, max(1, min(16, hi)), max(1, hi))
    return dict(op=op, B=B, max_len=max_len, max_new=min(max_new, max_len),
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]),
                page=rng.choice([8, 16, 24, 64, 128]), shape=rng.randrange(1, 1 << 30),
                Hq=Hkv * g, Hkv=Hkv, d=rng.choice([64, 128, 128]), atoms=_log(rng, 256, 32768))


def _lengths(case):
    """(tokens in the cache before the step, new tokens) of every request.
    shape 0: all alike; else mixed, idle requests and first tokens among them."""
    B, top, new = case["B"], case["max_len"], case["max_new"]
    if not case["shape"]:
        return [top - new] * B, [new] * B
    rng = random.Random(case["shape"])
    before, fresh = [], []
    for b in range(B):
        n = new if b == 0 or new == 1 else rng.choice([0, 1, rng.randint(1, new), new])
        whole = max(n, _log(rng, 1, top))
        if new == 1 and b and rng.random() < 0.05:
            n = 0
        before.append(whole - n)
        fresh.append(n)
    return before, fresh


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------------- states

def _codes(shape, atoms, gen):
    """Code words: uniform atoms, normal coefficients by falling magnitude."""
    idx = torch.randint(0, atoms, (*shape, K_ATOMS), generator=gen, device="cuda", dtype=torch.int32)
    c = torch.randn(*shape, K_ATOMS, generator=gen, device="cuda")
    c = c.gather(-1, c.abs().argsort(dim=-1, descending=True)).half()
    return (c.view(torch.int16).to(torch.int32) << 16) | idx


def _dictionary(atoms, d, gen):
    x = torch.randn(atoms, d, generator=gen, device="cuda")
    return (x / x.norm(dim=-1, keepdim=True)).to(torch.bfloat16)


def _tables(lens, page, n_pages, cols, gen):
    """A block table whose rows hold the requests' pages in a random order of
    the pool, -1 behind them, and the pages left over."""
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), cols), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        k = _pages(n, page)
        table[b, :k] = order[at:at + k]
        at += k
    return table, order[at:]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    page = case["page"]
    if case["op"] == "store":
        T, Hkv = case["T"], case["Hkv"]
        n_pages = _pages(T, page) + 2
        words = _codes((n_pages * page + 2 * T, Hkv), 32768, gen)
        old, k, v = words.split([n_pages * page, T, T])
        pages = torch.zeros(n_pages, Hkv, page, 2, K_ATOMS, dtype=torch.int32, device="cuda")
        pages[:, :, :, 0] = old.view(n_pages, page, Hkv, K_ATOMS).transpose(1, 2)
        slots = torch.randperm(n_pages, generator=gen, device="cuda")[:, None] * page
        slots = (slots + torch.arange(page, device="cuda")).view(-1)[:T].clone()
        slots[torch.rand(T, generator=gen, device="cuda") < 0.01] = -1    # padding of the step
        return dict(op="store", pages=pages, codes_k=k.contiguous(), codes_v=v.contiguous(),
                    slots=slots)
    before, new = _lengths(case)
    if case["op"] == "tables":
        used = sum(_pages(n, page) for n in before)
        need = sum(_pages(n + m, page) for n, m in zip(before, new))
        cols = _pages(case["max_len"], page) + 1
        table, free = _tables(before, page, need + 8, cols, gen)
        return dict(op="tables", lens=_i32(before), new=_i32(new), table=table, free=free.contiguous(),
                    n_free=_i32([need + 8 - used]), n_pages=need + 8, page=page,
                    T=max(1, sum(new)) + 3)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    lens = [n + m for n, m in zip(before, new)]
    n_pages = sum(_pages(n, page) for n in lens) + 1
    table, _ = _tables(lens, page, n_pages, _pages(case["max_len"], page), gen)
    T = sum(new)
    q = torch.randn(T, Hq, d, generator=gen, device="cuda") * 2
    q[:, :, torch.randperm(d, generator=gen, device="cuda")[:3]] *= 8     # a few strong channels
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    return dict(op="attend", q=q.to(torch.bfloat16), dk=_dictionary(case["atoms"], d, gen),
                dv=_dictionary(case["atoms"], d, gen),
                pages=_codes((n_pages, Hkv, page, 2), case["atoms"], gen), table=table,
                lens=_i32(lens), cu=_i32(cu), max_q=max(new), max_len=max(lens),
                total=sum(lens), window=case["window"], page=page)


# --------------------------------------------------------------- plain forms

def _plain_tables(s):
    P, lens, new = s["page"], s["lens"].long(), s["new"].long()
    table, free, n_free = s["table"], s["free"], s["n_free"].long()
    have, want = (lens + P - 1) // P, (lens + new + P - 1) // P
    fits = want <= table.shape[1]
    need = torch.where(fits, want - have, 0)
    upto = need.cumsum(0)
    fits = fits & (upto <= n_free)
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    col = torch.arange(table.shape[1], device="cuda")
    fresh = (col >= have[:, None]) & (col < want[:, None]) & fits[:, None]
    order = (upto - need)[:, None] + col - have[:, None]
    got = free[(n_free - 1 - order).clamp(0, free.shape[0] - 1)]
    table = torch.where(fresh, got, table)
    tok = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    there = b < lens.shape[0]
    b = b.clamp(max=lens.shape[0] - 1)
    pos = lens[b] + tok - cu[b]
    slot = table[b, (pos // P).clamp(max=table.shape[1] - 1)].long() * P + pos % P
    slot = torch.where(there & fits[b], slot, -1)
    return dict(table=table, slots=slot, cu=cu.int(), lens=torch.where(fits, lens + new, lens).int(),
                n_free=(n_free - torch.where(fits, need, 0).sum()).int())


def _plain_store(s):
    pages, slots = s["pages"], s["slots"]
    P = pages.shape[2]
    keep = slots >= 0
    page, off = slots[keep] // P, slots[keep] % P
    pages[page, :, off, 0] = s["codes_k"][keep]
    pages[page, :, off, 1] = s["codes_v"][keep]
    return pages


def _vectors(words, D):
    """The coded vectors of words [..., 16] in 32 bits."""
    c = (words >> 16).to(torch.int16).view(torch.float16).float()
    return (D.float()[(words & 0x7FFF).long()] * c.unsqueeze(-1)).sum(-2)


def _plain_attend(s):
    q, lens, cu, P, max_q = s["q"], s["lens"].long(), s["cu"].long(), s["page"], s["max_q"]
    T, Hq, d = q.shape
    Hkv = s["pages"].shape[1]
    B, g = lens.shape[0], Hq // Hkv
    t = torch.arange(s["max_len"], device="cuda")
    page = s["table"].long()[:, t // P].clamp(min=0)                    # [B, L]
    words = s["pages"][page, :, (t % P).expand(B, -1)]                  # [B, L, Hkv, 2, 16]
    K, V = _vectors(words[:, :, :, 0], s["dk"]), _vectors(words[:, :, :, 1], s["dv"])
    row = (cu[:-1, None] + torch.arange(max_q, device="cuda")).clamp(max=T - 1)
    x = q.float()[row].view(B, max_q, Hkv, g, d)
    sc = torch.einsum("bihgd,blhd->bhgil", x, K) / math.sqrt(d)
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(max_q, device="cuda")
    seen = (t <= pos[..., None]) & (t < lens[:, None, None])
    if s["window"]:
        seen = seen & (t > pos[..., None] - s["window"])
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    e = (sc - torch.where(top == -math.inf, 0.0, top)).exp()
    z = e.sum(-1, keepdim=True)
    e = e / torch.where(z == 0, 1.0, z)
    o = torch.einsum("bhgil,blhd->bihgd", e, V).reshape(B, max_q, Hq, d)
    tok = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    return o[b, tok - cu[b]].to(q.dtype)


# ----------------------------------------------------------- the package's

def _own_run(s):
    import sparse_dictionary_coded_b200 as sdk
    if s["op"] == "tables":
        if "ws" not in s:
            s["ws"] = sdk.new_workspace(sdk.sdk_block_tables_workspace_bytes(s["lens"].shape[0]))
        r = sdk.sdk_block_tables(s["lens"], s["new"], s["free"], s["n_free"], s["table"], s["page"],
                                 s["T"], n_pages=s["n_pages"], workspace=s["ws"])
        return dict(table=r.block_table, slots=r.slot_map, cu=r.cu_new, lens=r.new_lens,
                    n_free=r.n_free)
    if s["op"] == "store":
        if "ws" not in s:
            s["ws"] = sdk.new_workspace(sdk.sdk_paged_store_workspace_bytes())
        return sdk.sdk_paged_store(s["pages"], s["codes_k"], s["codes_v"], s["slots"],
                                   workspace=s["ws"])
    if "ws" not in s:
        s["ws"] = sdk.new_workspace(sdk.sdk_chunk_attn_workspace_bytes(
            s["lens"].shape[0], s["q"].shape[0], s["q"].shape[1], s["pages"].shape[1],
            s["q"].shape[2], s["dk"].shape[0], s["max_q"], s["max_len"], s["total"]))
    return sdk.sdk_chunk_attn(s["q"], s["dk"], s["dv"], s["pages"], s["table"], s["lens"], s["cu"],
                              s["max_q"], s["max_len"], total_len=s["total"], window=s["window"],
                              workspace=s["ws"])


def run(state):
    if own:
        return _own_run(state)
    return {"tables": _plain_tables, "store": _plain_store, "attend": _plain_attend}[state["op"]](state)


# --------------------------------------------------------------------- work

def work(case):
    page = case["page"]
    if case["op"] == "store":
        return {"bytes": case["T"] * (case["Hkv"] * 256 + 8), "flops": 0}
    before, new = _lengths(case)
    if case["op"] == "tables":
        fresh = sum(_pages(n + m, page) - _pages(n, page) for n, m in zip(before, new))
        # lengths and offsets, pages taken and entered, one old entry a request, slots
        return {"bytes": 20 * case["B"] + 8 * fresh + 8 * (max(1, sum(new)) + 3), "flops": 0}
    d, g = case["d"], case["Hq"] // case["Hkv"]
    pairs = tokens = 0
    for n, m in zip(before, new):
        w = case["window"] or n + m
        pairs += sum(min(n + i + 1, w) for i in range(m))
        tokens += min(n + m, w + m - 1) if m else 0
    coded = tokens * case["Hkv"]
    atoms = min(case["atoms"], coded * K_ATOMS)
    return {"bytes": coded * 128 + 2 * atoms * d * 2 + 2 * sum(new) * case["Hq"] * d * 2,
            # scores and weighted values of every pair, two vectors of 16 atoms a token
            "flops": pairs * case["Hq"] * 4 * d + coded * 2 * K_ATOMS * 2 * d}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """The attention in 64 bits, request by request and head by head; the
    other operators return whole numbers."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    before, new = _lengths(case)
    P, d, g = case["page"], case["d"], case["Hq"] // case["Hkv"]
    DK, DV = s["dk"].double(), s["dv"].double()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(before, new)):
        lo = max(0, n + 1 - case["window"]) if case["window"] else 0
        where = torch.arange(lo, n + m, device="cuda")
        for h in range(case["Hkv"] if m else 0):
            rec = s["pages"][s["table"][b].long()[where // P], h, where % P]
            kv = []
            for D, r in ((DK, rec[:, 0]), (DV, rec[:, 1])):
                x = torch.zeros(len(where), d, dtype=torch.float64, device="cuda")
                for j in range(K_ATOMS):
                    w = r[:, j]
                    c = torch.bitwise_right_shift(w, 16).to(torch.int16).view(torch.float16).double()
                    x += c[:, None] * D[(w % 32768).long()]
                kv.append(x)
            for i0 in range(0, m, 512):
                rows = s["q"][at + i0:at + min(m, i0 + 512), h * g:(h + 1) * g].double()
                sc = rows @ kv[0].T * d ** -0.5                         # [rows, g, tokens]
                place = n + i0 + torch.arange(rows.shape[0], device="cuda")[:, None, None]
                hidden = where > place
                if case["window"]:
                    hidden = hidden | (where <= place - case["window"])
                p = torch.softmax(sc.masked_fill(hidden, -math.inf), -1)
                out[at + i0:at + i0 + rows.shape[0], h * g:(h + 1) * g] = p @ kv[1]
        at += m
    return out
