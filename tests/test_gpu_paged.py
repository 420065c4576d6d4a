"""The paged code store on the GPU: plans, slot writes and chunk attention
against plain implementations in 64 bits.

Tolerance of the attention, per output element (derived, not fitted).  The
rebuilt vectors enter the products in fp16: |dK_d| <= u |K_d| + 2^-25 with
u = 2^-11, so a score is off by at most
    e_t = scale sum_d |q_d| (u |K_td| + 2^-25),
to which fp32 arithmetic adds at most (d + 40) 2^-23 times the sum of the
magnitudes it adds up (scores as sums over atoms included): with
    a_t = scale (sum_d |q_d| |K_td| + sum_j |c_tj| |<q, D_K[i_tj]>|)
    E = max over seen t of (u + (d + 40) 2^-23) a_t + scale 2^-25 sum_d |q_d|
(the second sum covers scores added up atom by atom with <q, D> in fp16).
Numerator and normaliser each change by a factor within exp(+-E); the
probability's and the value's fp16 roundings add u each, and the sums
2^-19 (values of V below 2^-14: 2^-25 absolute; weights per atom held in
fixed point: 2^-14 of the largest sum over atoms, covered by u).  So
    |out - ref| <= (exp(2E) - 1 + 3u + 2^-14) sum_t p_t sum_j |c_tj D_V| + 2^-8 |ref| + 2^-24.
"""

import math

import pytest
import torch

import sparse_dictionary_coded_b200 as sdk

pytestmark = pytest.mark.gpu
U = 2.0 ** -11


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _status(ws):
    rc, info = sdk.sdk_check_status(ws)
    return rc, info[1]


# ------------------------------------------------------------------- tables

def _tables_ref(lens, new, free, n_free, table, P, max_new, max_pages):
    table = [list(r) for r in table]
    row, taken, failed = 0, 0, False
    slots, cu, out = [-1] * max_new, [0], []
    for b, (n, m) in enumerate(zip(lens, new)):
        rows = max(m, 0)
        bad = n < 0 or m < 0 or n + m > 2 ** 31 - 1
        have = -(-n // P) if not bad else 0
        want = -(-(n + m) // P) if not bad else 0
        refused = bad or want > max_pages or (m > 0 and row + rows > max_new)
        if not refused:
            need = want - have
            if need and (failed or taken + need > n_free):
                refused = failed = True
        if not refused:
            for j in range(need):
                table[b][have + j] = free[n_free - 1 - taken - j]
            taken += need
            for i in range(m):
                slots[row + i] = table[b][(n + i) // P] * P + (n + i) % P
        row += rows
        cu.append(min(row, max_new))
        out.append(n if refused else n + m)
    return table, slots, cu, out, n_free - taken


def _tables_case(lens, new, P, max_pages, max_new, spare, seed=0, n_free=None):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    used = [max(0, -(-n // P)) if n < 2 ** 30 else 0 for n in lens]
    need = sum(max(0, -(-(n + max(m, 0)) // P) - u) if n < 2 ** 30 else 0
               for n, m, u in zip(lens, new, used))
    n_pages = sum(used) + need + spare + 1
    order = torch.randperm(n_pages, generator=g).tolist()
    table, at = [], 0
    for b in range(B):
        row = [-7] * max_pages
        k = min(used[b], max_pages)
        row[:k] = order[at:at + k]
        at += k
        table.append(row)
    free = order[at:]
    nf = max(0, need + spare) if n_free is None else n_free
    assert nf <= len(free)
    t = _i32(table)
    ws = sdk.new_workspace(sdk.sdk_block_tables_workspace_bytes(B))
    args = (_i32(lens), _i32(new), _i32(free), _i32([nf]), t, P, max_new)
    r = sdk.sdk_block_tables(*args, n_pages=n_pages, workspace=ws)
    want = _tables_ref(lens, new, free, nf, table, P, max_new, max_pages)
    st = _status(ws)
    for again in range(2):
        assert r.block_table.tolist() == want[0]
        assert r.slot_map.tolist() == want[1]
        assert r.cu_new.tolist() == want[2]
        assert r.new_lens.tolist() == want[3]
        assert r.n_free.tolist() == [want[4]]
        r = sdk.sdk_block_tables(*args, n_pages=n_pages, workspace=ws)   # the same plan again
    return st


@pytest.mark.parametrize("lens,new,P,max_pages,max_new", [
    ([0], [1], 16, 1, 1),
    ([0], [0], 16, 1, 5),                                   # nothing to do: all rows -1
    ([15, 16, 17, 0], [1, 1, 1, 0], 16, 2, 9),
    ([5, 0, 100, 31], [0, 7, 300, 1], 1, 400, 308),         # one-token pages
    ([5, 0, 100, 31], [0, 7, 300, 1], 7, 64, 310),
    ([1000, 3], [5000, 4000], 24, 251, 9000),               # several CTAs of slots
])
def test_tables(lens, new, P, max_pages, max_new):
    assert _tables_case(lens, new, P, max_pages, max_new, spare=3) == (0, 0)


@pytest.mark.parametrize("B", [1023, 1024, 1025, 4096])
def test_tables_many_requests(B):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 300, (B,), generator=g).tolist()
    new = torch.randint(0, 4, (B,), generator=g).tolist()
    assert _tables_case(lens, new, 16, 20, sum(new) + 2, spare=0, seed=B) == (0, 0)


def test_tables_refusals():
    # the pool runs out at the second request; the third needs no page and goes on
    st = _tables_case([16, 16, 20, 0], [1, 40, 3, 1], 16, 8, 45, spare=0, n_free=2)
    assert st[0] == 3
    # more pages than the table has columns: that request alone
    assert _tables_case([16, 16, 20], [1, 200, 13], 16, 4, 300, spare=4)[0] == 3
    # more tokens than the slot map has rows
    assert _tables_case([0, 0, 5], [10, 30, 0], 16, 4, 32, spare=4)[0] == 3
    # bad lengths
    assert _tables_case([-1, 8, 3], [4, -2, 1], 16, 4, 8, spare=4)[0] == 6
    assert _tables_case([2 ** 31 - 1, 8], [1, 1], 16, 4, 8, spare=4)[0] == 6
    # an empty stack, and requests that need nothing of it
    assert _tables_case([3, 0], [2, 0], 16, 4, 8, spare=0, n_free=0) == (0, 0)


def test_tables_bad_entries():
    """Pages out of range in the table, on the stack, and a stack counter
    past its end: recorded, the slots are -1, nothing is read behind."""
    ws = sdk.new_workspace(256)
    r = sdk.sdk_block_tables(_i32([3, 3]), _i32([1, 1]), _i32([0]), _i32([1]),
                             _i32([[99, -7], [1, -7]]), 16, 2, n_pages=4, workspace=ws)
    assert r.slot_map.tolist() == [-1, 19] and _status(ws)[0] == 6
    r = sdk.sdk_block_tables(_i32([0]), _i32([1]), _i32([50]), _i32([1]), _i32([[-7]]), 16, 1,
                             n_pages=4, workspace=ws)
    assert r.slot_map.tolist() == [-1] and r.block_table.tolist() == [[-1]]
    assert _status(ws)[0] == 6
    r = sdk.sdk_block_tables(_i32([0]), _i32([1]), _i32([2, 3]), _i32([9]), _i32([[-7]]), 16, 1,
                             n_pages=4, workspace=ws)
    assert r.block_table.tolist() == [[3]] and r.n_free.tolist() == [1]
    assert _status(ws)[0] == 6


# -------------------------------------------------------------------- store

def _words(shape, n, gen):
    idx = torch.randint(0, n, (*shape, 16), generator=gen, device="cuda", dtype=torch.int32)
    c = torch.randn(*shape, 16, generator=gen, device="cuda").half()
    return (c.view(torch.int16).to(torch.int32) << 16) | idx


@pytest.mark.parametrize("T,Hkv,P", [(1, 1, 1), (1, 8, 64), (37, 3, 7), (5000, 8, 16)])
def test_store(T, Hkv, P):
    g = torch.Generator(device="cuda").manual_seed(T)
    n_pages = T // P + 3
    pages = _words((n_pages, Hkv, P, 2), 1000, g)
    k, v = _words((T, Hkv), 1000, g), _words((T, Hkv), 1000, g)
    slots = torch.randperm(n_pages * P, generator=g, device="cuda")[:T]
    slots[torch.rand(T, generator=g, device="cuda") < 0.2] = -1
    want = pages.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s // P, :, s % P, 0] = k[t]
            want[s // P, :, s % P, 1] = v[t]
    ws = sdk.new_workspace(256)
    sdk.sdk_paged_store(pages, k, v.view(T * Hkv, 16), slots, workspace=ws)
    assert torch.equal(pages, want) and _status(ws)[0] == 0
    sdk.sdk_paged_store(pages, k, v, torch.full_like(slots, n_pages * P), workspace=ws)
    assert torch.equal(pages, want) and _status(ws)[0] == 6
    sdk.sdk_paged_store(pages, k[:0], v[:0], slots[:0], workspace=ws)
    assert torch.equal(pages, want) and _status(ws)[0] == 0


@pytest.mark.parametrize("T,Hkv,d,n,dtype", [
    (1, 8, 128, 32768, torch.bfloat16), (5, 8, 128, 4096, torch.float32),
    (9, 4, 64, 1000, torch.float32), (60, 3, 64, 1000, torch.bfloat16)])
def test_append(T, Hkv, d, n, dtype):
    """The words of sdk_encode in the slots, whichever encoder runs."""
    g = torch.Generator(device="cuda").manual_seed(T)
    D = torch.nn.functional.normalize(
        torch.randn(2, n, d, generator=g, device="cuda"), dim=-1).to(torch.bfloat16)
    x = torch.randn(2, T, Hkv, d, generator=g, device="cuda").to(dtype)
    P = 16
    pages = torch.zeros(T // P + 2, Hkv, P, 2, 16, dtype=torch.int32, device="cuda")
    slots = torch.randperm(pages.shape[0] * P, generator=g, device="cuda")[:T]
    slots[0] = -1 if T > 1 else slots[0]
    ws = sdk.sdk_paged_append(pages, x[0], x[1], D[0].contiguous(), D[1].contiguous(), slots)
    assert _status(ws)[0] == 0
    want = torch.zeros_like(pages)
    for s in range(2):
        w = sdk.sdk_encode(x[s], D[s].contiguous()).view(T, Hkv, 16)
        for t, at in enumerate(slots.tolist()):
            if at >= 0:
                want[at // P, :, at % P, s] = w[t]
    assert torch.equal(pages, want)


# ---------------------------------------------------------------- attention

def _vec(words, D):
    c = (words >> 16).to(torch.int16).view(torch.float16).double()
    i = (words & 0x7FFF).long()
    return c, i, (c[..., None] * D.double()[i]).sum(-2)


def _attend_ref(q, dk, dv, pages, table, lens, cu, causal, window, scale):
    """(out, tolerance, lse, lse tolerance) in 64 bits, request by request."""
    T, Hq, d = q.shape
    Hkv, P = pages.shape[1:3]
    g = Hq // Hkv
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    tol, lse = torch.zeros_like(out), torch.full((T, Hq), -math.inf, dtype=torch.float64,
                                                 device="cuda")
    etol = torch.zeros_like(lse)
    for b in range(len(lens)):
        r0, r1, L = cu[b], cu[b + 1], lens[b]
        if r1 == r0 or L == 0:
            continue
        t = torch.arange(L, device="cuda")
        rec = pages[table[b].long()[t // P], :, t % P]                 # [L, Hkv, 2, 16]
        ck, ik, K = _vec(rec[:, :, 0], dk)
        cv, iv, V = _vec(rec[:, :, 1], dv)
        Vabs = (cv.abs()[..., None] * dv.double().abs()[iv]).sum(-2)
        x = q[r0:r1].double()
        pos = (L - (r1 - r0) + torch.arange(r1 - r0, device="cuda"))[:, None]
        seen = torch.ones(r1 - r0, L, dtype=torch.bool, device="cuda")
        if causal:
            seen = t <= pos
        if window:
            seen = seen & (t > pos - window)
        for hq in range(Hq):
            h = hq // g
            xq = x[:, hq]
            s = (xq @ K[:, h].T * scale).masked_fill(~seen, -math.inf)
            qd = xq @ dk.double().T                                    # [rows, atoms]
            atoms = torch.zeros_like(s)
            for j in range(16):
                atoms += ck[:, h, j].abs() * qd.abs()[:, ik[:, h, j]]
            a = scale * (xq.abs() @ K[:, h].abs().T + atoms)
            E = ((U + (d + 40) * 2.0 ** -23) * a).masked_fill(~seen, 0.0).amax(-1) \
                + scale * 2.0 ** -25 * xq.abs().sum(-1)
            any_ = seen.any(-1)
            p = torch.softmax(torch.where(any_[:, None], s, 0.0), -1) * any_[:, None]
            o = p @ V[:, h]
            out[r0:r1, hq] = o
            tol[r0:r1, hq] = (torch.expm1(2 * E)[:, None] + 3 * U + 2.0 ** -14) * (p @ Vabs[:, h]) \
                + 2.0 ** -8 * o.abs() + 2.0 ** -24
            lse[r0:r1, hq] = torch.logsumexp(s, -1)
            etol[r0:r1, hq] = E + 2.0 ** -16 * (1 + lse[r0:r1, hq].abs().nan_to_num(posinf=0))
    return out, tol, lse, etol


class Case:
    """Requests with `lens` tokens, the last `new` of them new, on random
    pages; unused slots and pages hold words that no call may use."""

    def __init__(self, lens, new, Hq=8, Hkv=2, d=128, n=3000, P=16, seed=0, q_scale=2.0, cols=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.new, self.P = lens, new, P
        used = [-(-x // P) for x in lens]
        n_pages = sum(used) + 2
        self.pages = torch.full((n_pages, Hkv, P, 2, 16), 0x7E007FFF, dtype=torch.int32,
                                device="cuda")      # a NaN coefficient of atom 32767
        order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        cols = cols or max(max(used), 1)
        table, at = [], 0
        for b, L in enumerate(lens):
            ids = order[at:at + used[b]]
            at += used[b]
            table.append(ids + [-5] * (cols - used[b]))
            for c, pg in enumerate(ids):
                k = min(P, L - c * P)
                self.pages[pg, :, :k] = _words((Hkv, k, 2), n, g)
        self.table = _i32(table)
        self.cu = [0]
        for m in new:
            self.cu.append(self.cu[-1] + m)
        D = torch.randn(2, n, d, generator=g, device="cuda")
        D = (D / D.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
        self.dk, self.dv = D[0].contiguous(), D[1].contiguous()
        self.q = (torch.randn(self.cu[-1], Hq, d, generator=g, device="cuda") * q_scale).to(
            torch.bfloat16)

    def run(self, causal=True, window=0, ws=None, max_q=None, max_len=None, total=None, q=None,
            **kw):
        max_len = max_len or max(max(self.lens), 1)
        max_len = min(max_len, self.table.shape[1] * self.P)
        return sdk.sdk_chunk_attn(
            self.q if q is None else q, self.dk, self.dv, self.pages, self.table, _i32(self.lens),
            _i32(self.cu), max_q or max(max(self.new), 1), max_len,
            total_len=sum(self.lens) if total is None else total, causal=causal, window=window,
            workspace=ws, **kw)

    def workspace(self, max_q=None, max_len=None, total=None):
        T, Hq, d = self.q.shape
        return sdk.new_workspace(sdk.sdk_chunk_attn_workspace_bytes(
            len(self.lens), T, Hq, self.pages.shape[1], d, self.dk.shape[0],
            max_q or max(max(self.new), 1), max_len or max(max(self.lens), 1),
            sum(self.lens) if total is None else total))

    def check(self, causal=True, window=0, scale=None, **bounds):
        T, Hq, d = self.q.shape
        ws = self.workspace(**bounds)
        lse = torch.full((T, Hq), 77.0, device="cuda")
        out = self.run(causal, window, ws, lse=lse, scale=scale, **bounds)
        assert _status(ws) == (0, 0)
        want, tol, wl, el = _attend_ref(self.q, self.dk, self.dv, self.pages, self.table, self.lens,
                                        self.cu, causal, window, scale or 1 / math.sqrt(d))
        far = (out.double() - want).abs() - tol
        assert not (far > 0).any() and torch.isfinite(out).all(), "over by %g" % far.max().item()
        empty = wl == -math.inf
        assert torch.equal(lse == -math.inf, empty)
        assert ((lse.double() - wl).abs()[~empty] <= el[~empty]).all()
        return out


SHAPES = [
    dict(lens=[1], new=[1]),                                          # one token sees itself
    dict(lens=[2], new=[2], Hq=1, Hkv=1, d=64, n=1, P=1),             # one atom, one-token pages
    dict(lens=[127, 128, 129, 1], new=[1, 1, 1, 1]),                  # single tokens, tile edges
    dict(lens=[300, 40, 0, 513], new=[3, 0, 0, 5], P=24),             # drafts, idle, empty
    dict(lens=[130], new=[130], Hq=4, Hkv=1, d=64, P=64),             # a whole prompt
    dict(lens=[257, 600], new=[257, 200], Hq=6, Hkv=2, P=7),          # g = 3, pages inside tiles
    dict(lens=[700], new=[129], Hq=5, Hkv=1, P=100),                  # g = 5
    dict(lens=[400, 1000], new=[64, 33], Hq=8, Hkv=8, d=64),          # g = 1
    dict(lens=[5000], new=[1], Hq=32, Hkv=8, n=32768, P=64),          # one long step
    dict(lens=[2100, 1900, 35], new=[1, 2, 1], Hq=8, Hkv=2, n=32768), # few rows, several splits
    dict(lens=[1500], new=[700], Hq=16, Hkv=1, P=128),                # g = 16
    dict(lens=[4096], new=[2], Hq=64, Hkv=1, d=64, n=1001),           # g = 64, odd atom count
    dict(lens=[9000], new=[1], Hq=32, Hkv=8, n=32768, P=64),          # few rows, long contexts:
    dict(lens=[20001, 0, 500, 1], new=[3, 0, 2, 1], Hq=12, Hkv=4, n=1001, P=24, d=64),
    dict(lens=[70000, 3], new=[1, 1], Hq=1, Hkv=1, n=32767, P=7),     # one row of a pair
    dict(lens=[1100] * 30, new=[1] * 30, Hq=4, Hkv=2, n=513, d=64),   # many requests
    dict(lens=[150000], new=[1], Hq=3, Hkv=1, n=2, P=64),             # two atoms
    dict(lens=[9000, 5, 1300], new=[40, 5, 100], Hq=4, Hkv=1, n=300, d=64, P=24),  # blocks in parts
    dict(lens=[1500] * 40, new=[30] * 40, Hq=8, Hkv=4, n=300, d=64, P=16),   # equal shares of them
    dict(lens=[700, 0, 90, 30] * 20, new=[3, 0, 2, 1] * 20, Hq=6, Hkv=3, n=400, P=8),  # many requests in one pass
    dict(lens=[2000, 17, 16, 33], new=[8, 8, 1, 4], Hq=4, Hkv=1, n=300, P=16),   # 32 rows in one pass
    dict(lens=[33000, 100], new=[40, 2], Hq=4, Hkv=1, P=32),          # one block shared by all SMs
    dict(lens=[2500], new=[2500], Hq=32, Hkv=8, n=300, d=64, P=64),   # more blocks than SMs
]


@pytest.mark.parametrize("kw", SHAPES, ids=lambda k: "%s-%s" % (k["lens"], k["new"]))
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 50)])
def test_attend(kw, causal, window):
    Case(**kw, seed=3).check(causal, window)


@pytest.mark.parametrize("scale,q_scale", [(0.01, 1.0), (1.0, 2.0), (0.3, 30.0), (0.0884, 1e-30)])
def test_attend_scales(scale, q_scale):
    """Flat and one-hot softmaxes, and queries far below fp16's range."""
    Case([200, 3000], [70, 1], seed=5, q_scale=q_scale).check(scale=scale)


def test_attend_more_new_than_context():
    """Rows before the context's first token see nothing: zeros, lse -inf."""
    c = Case([5, 0], [9, 3], seed=1)
    out = c.check()
    assert out[:4].abs().max() == 0 and out[9:].abs().max() == 0 and out[4:9].abs().min(-1)[0].max() > 0


def test_rows_behind_the_last_request_stay():
    c = Case([300, 50], [20, 1], seed=2)
    out = torch.full((40, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((40, 8), 5.0, device="cuda")
    q = torch.zeros_like(out)
    q[:21] = c.q
    q[21:] = float("nan")
    got = c.run(q=q, out=out, lse=lse)
    assert torch.equal(got[:21], c.run()) and (got[21:] == 3.0).all() and (lse[21:] == 5.0).all()


@pytest.mark.parametrize("lens,new", [([400], [300]), ([3000], [2]), ([260, 50], [1, 50]),
                                      ([40000, 50], [3, 1])])
def test_bad_words_in_masked_places(lens, new):
    """NaN and infinite coefficients and atoms past the dictionary in tokens
    that only the last row sees: recorded, every other row is as before."""
    c = Case(lens, new, seed=4)
    want = c.run()
    b = 0
    t = lens[b] - 1
    page = c.table[b, t // c.P].item()
    for word in (0x7E000001, 0x7C000001, -0x03FFFFFF, 0x3C007FFF):     # NaN, inf, -inf, atom 32767
        c.pages[page, :, t % c.P, :, 3] = word
        ws = c.workspace()
        got = c.run(ws=ws)
        assert _status(ws)[0] == 6
        last = c.cu[b + 1] - 1
        keep = [r for r in range(got.shape[0]) if r != last]
        assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("lens,new,i", [([500, 900], [140, 1], 70), ([40000, 900], [3, 1], 1)])
def test_bad_query_rows_stay_alone(lens, new, i):
    c = Case(lens, new, seed=6)
    want = c.run()
    c.q[2, 2] = float("nan")
    c.q[i, 5, 7] = float("inf")
    got = c.run()
    bad = torch.zeros(got.shape[:2], dtype=torch.bool, device="cuda")
    bad[2, 2] = bad[i, 5] = True
    assert torch.equal(got[~bad], want[~bad])
    assert torch.isnan(got[2, 2]).all() and torch.isnan(got[i, 5]).all()


def test_few_rows_refusals():
    """Refusals and bad pages on the long-context form.  (Refusing a request
    cuts the others' contexts at other places: equal within the tolerance.)"""
    c = Case([50000, 30000], [2, 1], Hkv=2, Hq=4, seed=7)
    T, Hq, d = c.q.shape
    ref, tol, _, _ = _attend_ref(c.q, c.dk, c.dv, c.pages, c.table, c.lens, c.cu, True, 0,
                                 1 / math.sqrt(d))
    near = lambda out, rows: ((out.double() - ref).abs() <= tol)[rows].all()
    ws = c.workspace()

    def go(status, kept, left, **kw):
        out = torch.full_like(c.q, 9.0)
        c.run(ws=ws, out=out, **kw)
        assert _status(ws)[0] == status and near(out, kept) and (out[left] == 9.0).all()

    a, b = slice(0, 2), slice(2, 3)
    go(3, b, a, max_len=40000)
    # room for 2 pairs (two tokens, two heads a group) x 2 KV heads x 50000
    # tokens: request 0 takes it all
    go(3, a, b, total=50000)
    c.lens = [50000, -4]
    go(6, a, b, total=80000)
    c.lens = [50000, 30000]
    want = c.run()
    c.table[0, 7] = -1
    out = c.run(ws=ws)
    assert _status(ws)[0] == 6 and torch.equal(out[b], want[b])


@pytest.mark.parametrize("size", [1e-5, 1.0, 3e3])
def test_few_rows_value_sizes(size):
    """Value coefficients of any size, and one token a thousand times the
    others (the fixed point of the weights follows the sums)."""
    c = Case([40000], [1], Hq=4, Hkv=2, n=5000, seed=11)
    w = c.pages[:, :, :, 1]
    coef = (w >> 16).to(torch.int16).view(torch.float16).float() * size
    coef[5, :, 3] *= 1000.0 if size < 100 else 10.0
    coef = coef.clamp(-65504, 65504)           # as words are made (include/sdk.h)
    good = (w & 0x7FFF) < 5000
    c.pages[:, :, :, 1] = torch.where(
        good, (coef.half().view(torch.int16).to(torch.int32) << 16) | (w & 0x7FFF), w)
    c.check()


def test_refused_requests():
    """A request outside its bounds is recorded and not written; the others
    are as without it."""
    c = Case([300, 200, 100], [10, 20, 5], seed=7)
    want = c.run()
    ws = c.workspace()

    def go(status, keep, **kw):
        out = torch.full_like(c.q, 9.0)
        c.run(ws=ws, out=out, **kw)
        assert _status(ws)[0] == status
        for b in range(3):
            rows = slice(c.cu[b], c.cu[b + 1])
            if b in keep:
                assert torch.equal(out[rows], want[rows]), b
            else:
                assert (out[rows] == 9.0).all(), b

    go(0, [0, 1, 2])
    go(3, [0, 2], max_q=15)
    go(3, [1, 2], max_len=250)
    # room for 300 // 128 + 3 = 5 tiles; the requests take 3, 2 and 1
    go(3, [0, 1], total=300)
    lens = c.lens
    c.lens = [300, -1, 100]
    go(6, [0, 2])
    c.lens = lens
    cu = c.cu
    out = torch.full_like(c.q, 9.0)
    c.cu = [0, 10, 5, 35]                     # falls: requests 1 (and its rows) cannot be read
    c.run(ws=ws, out=out)
    assert _status(ws)[0] == 6 and torch.equal(out[:10][:5], want[:5])
    c.cu = [0, 10, 30, 36]                    # past the rows of q
    out = torch.full_like(c.q, 9.0)
    c.run(ws=ws, out=out)
    assert _status(ws)[0] == 6 and torch.equal(out[:30], want[:30]) and (out[30:] == 9.0).all()
    c.cu = cu
    c.table[1, 3] = c.pages.shape[0]          # a page past the pool: its tokens count as zero vectors
    out = c.run(ws=ws)
    assert _status(ws)[0] == 6 and torch.equal(out[:10], want[:10]) and torch.equal(out[30:], want[30:])


def test_offsets_past_32_bits():
    """Pages at the far end of a pool of more than 2^31 words (10 GB)."""
    c = Case([150, 700], [3, 1], seed=8)
    want = c.run()
    n, extra = c.pages.shape[0], (2 ** 31 // (2 * 16 * 32)) + 1000
    big = torch.empty(extra + n, 2, c.P, 2, 16, dtype=torch.int32, device="cuda")
    assert big.numel() > 2 ** 31
    big[extra:] = c.pages
    c.pages, c.table = big, torch.where(c.table >= 0, c.table + extra, c.table)
    assert torch.equal(c.run(), want)
    k = _words((2, 2), 100, torch.Generator(device="cuda").manual_seed(1))
    slots = torch.tensor([(extra + n) * c.P - 1, extra * c.P], device="cuda")
    sdk.sdk_paged_store(big, k, k, slots)
    assert torch.equal(big[-1, :, -1, 0], k[0]) and torch.equal(big[extra, :, 0, 1], k[1])


@pytest.mark.parametrize("lens,new", [([2500, 300], [4, 200]), ([40000, 300], [2, 1]),
                                      ([30000, 300], [40, 30])])
def test_other_stream_and_repeat(lens, new):
    """The same bits on another stream, with a workspace of old contents."""
    c = Case(lens, new, seed=9)
    want = c.run()
    ws = c.workspace()
    ws[256:] = 0xFF
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = c.run(ws=ws)
        b = c.run(ws=ws)
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


@pytest.mark.parametrize("size", [1e-3, 30.0])
@pytest.mark.parametrize("lens,new", [([900, 300], [50, 1]), ([40000], [1])])
def test_dictionaries_of_other_norms(size, lens, new):
    c = Case(lens, new, seed=12)
    c.dk, c.dv = (c.dk * size).contiguous(), (c.dv * size).contiguous()
    c.check(scale=1 / math.sqrt(128) / size)


@pytest.mark.parametrize("lens,new", [([900, 300], [50, 1]), ([40000], [1])])
def test_entries_out_of_range_are_recorded(lens, new):
    """Rebuilt entries, or <q, D_K>, past fp16's range: recorded, and finite."""
    c = Case(lens, new, seed=13)
    c.dk, c.dv = (c.dk * 1e6).contiguous(), (c.dv * 1e6).contiguous()
    ws = c.workspace()
    assert torch.isfinite(c.run(ws=ws, scale=1e-9)).all() and _status(ws)[0] == 6


@pytest.mark.parametrize("kw", SHAPES, ids=lambda k: "%s-%s" % (k["lens"][:4], k["new"][:4]))
def test_nothing_is_written_behind_the_workspace(kw):
    c = Case(**kw, seed=14)
    n = c.workspace().numel()
    ws = sdk.new_workspace(n + (1 << 20))
    ws[n:] = 0xA5
    out = torch.full((c.q.shape[0] + 3, *c.q.shape[1:]), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(ws=ws[:n], out=out[1:-2])
    assert (ws[n:] == 0xA5).all() and (out[0] == 7.0).all() and (out[-2:] == 7.0).all()
    with pytest.raises(sdk.SdkError, match="SDK_ERR_CAPACITY"):
        c.run(ws=ws[:(n - 1) // 256 * 256])


def test_offsets_that_fall_stay_inside():
    """cu_q going up and down claims rows many times over: requests are
    refused where the workspace has no room for them, nothing else is hurt."""
    c = Case([200] * 40, [10] * 40, Hq=8, Hkv=2, n=500)
    n = c.workspace().numel()
    ws = sdk.new_workspace(n + (1 << 20))
    ws[n:] = 0xA5
    c.cu = [0 if i % 2 else 10 for i in range(41)]
    c.run(ws=ws[:n])
    assert _status(ws)[0] in (3, 6) and (ws[n:] == 0xA5).all()
    c.cu = [0] + [400 - 10 * (i % 40) for i in range(40)]
    c.run(ws=ws[:n])
    assert _status(ws)[0] in (3, 6) and (ws[n:] == 0xA5).all()


@pytest.mark.parametrize("bounds", [dict(max_len=600), dict(max_len=4096, total=0),
                                    dict(max_len=65536, total=0), dict(max_q=64, max_len=600, total=0),
                                    dict(max_q=64, max_len=65536, total=0)], ids=str)
@pytest.mark.parametrize("new", [[1, 1, 0, 1], [3, 17, 0, 2], [60, 17, 0, 2]])
@pytest.mark.parametrize("window", [0, 50])
def test_loose_bounds(new, bounds, window):
    """Bounds far above the lengths choose another form, not another result."""
    Case([300, 17, 0, 600], new, n=2000, cols=4096, seed=18).check(window=window, **bounds)


def test_many_requests():
    """4096 requests of a few tokens, idle ones among them."""
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 12, (4096,), generator=g).tolist()
    new = [min(x, 1 + i % 2) if i % 7 else 0 for i, x in enumerate(lens)]
    Case(lens, new, Hq=2, Hkv=1, d=64, n=100, P=4, cols=3).check()


def test_two_calls_at_once():
    """Two calls on two streams with a workspace each."""
    a, b = Case([3000], [300], seed=15), Case([30000], [1], seed=16)
    want = [a.run(), b.run()]
    ws, streams = [a.workspace(), b.workspace()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.run(ws=ws[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


def test_stream_argument():
    """A call given a stream runs, and makes its outputs, on that stream."""
    c = Case([700], [5], seed=17)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    r = sdk.sdk_block_tables(_i32([3]), _i32([2]), _i32([1, 0]), _i32([2]), _i32([[0, -1]]), 4, 2,
                             stream=s)
    s.synchronize()
    assert r.slot_map.tolist() == [3, 0] and r.n_free.tolist() == [1]


def test_arguments_are_checked():
    c = Case([20], [2])
    with pytest.raises(ValueError, match="dtype"):
        c.run(q=c.q.float())
    with pytest.raises(ValueError, match="contiguous"):
        c.run(q=c.q.expand(2, 8, 128)[:, ::2])
    with pytest.raises(ValueError, match="CUDA tensor"):
        c.run(q=c.q.cpu())
    with pytest.raises(ValueError, match="shape"):
        c.run(out=c.q[:1])
    with pytest.raises(ValueError, match="cu_q"):
        sdk.sdk_chunk_attn(c.q, c.dk, c.dv, c.pages, c.table, _i32([20, 20]), _i32([0, 2]), 2, 32)
    with pytest.raises(sdk.SdkError, match="SDK_ERR_INVALID_ARG"):
        c.run(window=-1)
    with pytest.raises(ValueError, match="32 bits"):
        c.run(max_q=1 << 40)
    with pytest.raises(ValueError, match="n_new"):
        sdk.sdk_block_tables(_i32([3]), _i32([2, 2]), _i32([1]), _i32([1]), _i32([[0]]), 4, 2)
    with pytest.raises(ValueError, match="pages must be"):
        sdk.sdk_paged_store(c.pages[0], c.table, c.table, torch.zeros(1, device="cuda").long())


# ------------------------------------------------------------ all together

class _Serving:
    """A small serving loop over three requests, all plans on the device."""

    def __init__(self, seed=0, Hq=8, Hkv=2, d=64, n=500, P=8):
        g = torch.Generator(device="cuda").manual_seed(seed)
        D = torch.randn(2, n, d, generator=g, device="cuda")
        D = (D / D.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
        self.dk, self.dv = D[0].contiguous(), D[1].contiguous()
        self.store = sdk.PagedCodeStore(64, Hkv, P)
        self.table = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
        self.lens = _i32([0, 0, 0])
        self.g, self.Hq, self.Hkv, self.d = g, Hq, Hkv, d

    def vectors(self, T):
        r = lambda h: torch.randn(T, h, self.d, generator=self.g, device="cuda").to(torch.bfloat16)
        return r(self.Hq), r(self.Hkv), r(self.Hkv)

    def step(self, new, q, k, v):
        plan = self.store.plan(self.lens, new, self.table, q.shape[0])
        sdk.sdk_paged_append(self.store.pages, k, v, self.dk, self.dv, plan.slot_map)
        out = sdk.sdk_chunk_attn(q, self.dk, self.dv, self.store.pages, self.table, plan.new_lens,
                                 plan.cu_new, q.shape[0], 160)
        self.lens = plan.new_lens
        return out, plan


def test_serving_steps():
    """Prompts, a step of single tokens, a piece and a draft: the paged
    answers against attention in 64 bits over the codes of every vector so
    far; then a finished request's pages serve another."""
    s = _Serving()
    hist = [[], [], []]
    for new in ([30, 0, 7], [1, 0, 1], [5, 60, 1], [1, 1, 1]):
        q, k, v = s.vectors(sum(new))
        out, plan = s.step(_i32(new), q, k, v)
        kw, vw = (sdk.sdk_encode(x, D).view(-1, s.Hkv, 16) for x, D in ((k, s.dk), (v, s.dv)))
        at = 0
        for b, m in enumerate(new):
            hist[b] += list(zip(kw[at:at + m], vw[at:at + m]))
            at += m
        assert plan.new_lens.tolist() == [len(x) for x in hist]
        # a plain store of the same codes: one page per request
        L = max(len(x) for x in hist)
        flat = torch.zeros(3, s.Hkv, L, 2, 16, dtype=torch.int32, device="cuda")
        for b, x in enumerate(hist):
            for t, (a, c) in enumerate(x):
                flat[b, :, t, 0], flat[b, :, t, 1] = a, c
        want, tol, _, _ = _attend_ref(q, s.dk, s.dv, flat, _i32([[0], [1], [2]]),
                                      plan.new_lens.tolist(), plan.cu_new.tolist(), True, 0,
                                      1 / math.sqrt(s.d))
        assert ((out.double() - want).abs() <= tol).all()
    before = s.store.n_free.item()
    used = -(-len(hist[1]) // 8)
    s.store.release(s.table[1, :used].clone())
    assert s.store.n_free.item() == before + used
    s.lens = s.lens * _i32([1, 0, 1])
    q, k, v = s.vectors(9)
    _, plan = s.step(_i32([0, 9, 0]), q, k, v)
    assert plan.new_lens.tolist()[1] == 9 and plan.n_free.tolist() == [before + used - 2]
    live = [p for b, x in enumerate(plan.new_lens.tolist()) for p in s.table[b, :-(-x // 8)].tolist()]
    assert len(set(live)) == len(live)


@pytest.mark.parametrize("P", [1, 3, 64])
@pytest.mark.parametrize("shift", [0, 1])
def test_many_rows(P, shift):
    """Slots of thousands of rows: idle requests, requests of one and of many
    rows, refused ones, a map at an odd address and of an odd length."""
    g = torch.Generator().manual_seed(P)
    lens = torch.randint(0, 50, (300,), generator=g).tolist()
    new = [0 if i % 5 == 0 else 1 if i % 5 == 1 else int(torch.randint(1, 90, (1,), generator=g))
           for i in range(300)]
    lens[7], new[299] = -1, 1 << 30                      # refused
    cols = 200
    have = [max(-(-x // P), 0) for x in lens]
    pool = sum(-(-(x + n) // P) for x, n in zip(lens, new) if 0 <= x and n < 1 << 20)
    table = torch.full((300, cols), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(have):
        table[b, :k] = torch.arange(at, at + k)
        at += k
    free = list(range(at, pool))[::-1]
    max_new = sum(n for n in new if n < 1 << 20) + 1001
    # what is wanted, request by request (the last one passes max_new)
    want, pos, over, k, asked = [], 0, False, 0, 0
    for b in range(300):
        pos += max(new[b], 0)
        over = pos > max_new
        if lens[b] < 0 or over:
            want += [-1] * (0 if over else new[b])
            continue
        # (request 299's own pages are not among those of the pool that the
        # step asks for: the last pages are missing, and a request that needs
        # one is refused)
        need = -(-(lens[b] + new[b]) // P) - have[b]
        asked += need
        if need > 0 and asked > len(free):
            want += [-1] * new[b]
            continue
        pages = table[b, :have[b]].tolist()
        while len(pages) * P < lens[b] + new[b]:
            pages.append(free[len(free) - 1 - k])
            k += 1
        want += [pages[t // P] * P + t % P for t in range(lens[b], lens[b] + new[b])]
    want += [-1] * (max_new - len(want))
    room = torch.full((max_new + 2,), 77, dtype=torch.int64, device="cuda")
    out = room[shift:shift + max_new]
    r = sdk.sdk_block_tables(_i32(lens), _i32(new), _i32(free), _i32([len(free)]), table.cuda(), P,
                             max_new, n_pages=pool, slot_map=out)
    assert r.slot_map.tolist() == want and r.n_free.tolist() == [len(free) - k]
    assert room[:shift].tolist() == [77] * shift and room[shift + max_new:].tolist() == [77] * (2 - shift)


@pytest.mark.parametrize("given", [(), ("slot_map",), ("cu_new", "n_free_out"), ("new_lens",)])
def test_outputs_given_or_new(given):
    """New outputs do not overlap each other, given ones are the ones returned."""
    new = dict(slot_map=torch.full((7,), 99, device="cuda"), cu_new=_i32([9] * 4),
               new_lens=_i32([9] * 3), n_free_out=_i32([9]))
    r = sdk.sdk_block_tables(_i32([3, 0, 5]), _i32([2, 0, 3]), _i32([5, 4, 3, 2, 1, 0]), _i32([4]),
                             _i32([[0, -1, -1], [-1] * 3, [4, 5, -1]]), 4, 7,
                             **{k: new[k] for k in given})
    got = dict(slot_map=r.slot_map, cu_new=r.cu_new, new_lens=r.new_lens, n_free_out=r.n_free)
    assert all(got[k] is new[k] or got[k].data_ptr() == new[k].data_ptr() for k in given)
    # request 0 takes page 2 (top of four), request 2 fills page 5: 5 + 3 = 8 tokens
    assert r.block_table.tolist() == [[0, 2, -1], [-1] * 3, [4, 5, -1]]
    assert r.slot_map.tolist() == [3, 8, 21, 22, 23, -1, -1]
    assert r.cu_new.tolist() == [0, 2, 2, 5] and r.new_lens.tolist() == [5, 0, 8]
    assert r.n_free.tolist() == [3]
    for k, t in got.items():
        t.zero_()
        assert all(o is t or o.numel() == 0 or (o == 0).all() or k != n for n, o in got.items())


def test_pages_released_twice_are_dropped():
    """What the stack has no place for is dropped; the stack stays where a
    captured plan reads it."""
    store = sdk.PagedCodeStore(6, 1, 4)
    at = store.free_pages.data_ptr()
    table = _i32([[-1] * 6])
    store.plan(_i32([0]), _i32([12]), table, 12)
    store.release(_i32([0, 1, 2]))
    assert store.n_free.tolist() == [6] and sorted(store.free_pages.tolist()) == list(range(6))
    store.release(_i32([0, 1]))
    assert store.n_free.tolist() == [6] and sorted(store.free_pages.tolist()) == list(range(6))
    assert store.free_pages.data_ptr() == at


def test_captured_step_replays():
    """One step of single tokens captured in a CUDA graph and replayed: the
    lengths advance on the device, and every replay equals the eager step."""
    a, b = _Serving(seed=3), _Serving(seed=3)
    first = _i32([30, 40, 3])
    q, k, v = a.vectors(73)
    b.vectors(73)
    a.step(first, q, k, v)
    b.step(first, q, k, v)
    ones = _i32([1, 1, 1])
    q, k, v = (x.clone() for x in b.vectors(3))
    lens, n_free = b.lens.clone(), b.store.n_free.clone()
    st = dict(ws_t=sdk.new_workspace(256),
              ws_a=sdk.new_workspace(sdk.sdk_paged_append_workspace_bytes(3, 2, 64, 500)),
              ws_c=sdk.new_workspace(sdk.sdk_chunk_attn_workspace_bytes(3, 3, 8, 2, 64, 500, 1, 160)))
    out = torch.zeros_like(q)

    def step():
        plan = sdk.sdk_block_tables(lens, ones, b.store.free_pages, n_free, b.table, 8, 3,
                                    workspace=st["ws_t"])
        sdk.sdk_paged_append(b.store.pages, k, v, b.dk, b.dv, plan.slot_map, workspace=st["ws_a"])
        sdk.sdk_chunk_attn(q, b.dk, b.dv, b.store.pages, b.table, plan.new_lens, plan.cu_new, 1,
                           160, workspace=st["ws_c"], out=out)
        lens.copy_(plan.new_lens)
        n_free.copy_(plan.n_free)

    keep = [t.clone() for t in (lens, n_free, b.table, b.store.pages)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                   # before the capture: attributes, modules
    torch.cuda.current_stream().wait_stream(side)
    for t, o in zip((lens, n_free, b.table, b.store.pages), keep):
        t.copy_(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        x = a.vectors(3)
        for t, o in zip((q, k, v), x):
            t.copy_(o)
        graph.replay()
        want, _ = a.step(ones, *x)
        assert torch.equal(out, want)
        assert torch.equal(lens, a.lens) and torch.equal(n_free, a.store.n_free)
    for name in ("ws_t", "ws_a", "ws_c"):
        assert _status(st[name])[0] == 0
