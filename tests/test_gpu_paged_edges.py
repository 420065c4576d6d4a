"""Chunk attention and plans where they can go wrong: work smaller than the
launch, NaN under short windows, pages freed behind a window, weights of very
different sizes, flat attention over long contexts, captured plans.  The plain
implementations and the tolerances are those of test_gpu_paged.py; where a test
needs its own, it stands beside it."""

import math

import pytest
import torch

import sparse_dictionary_coded_b200 as sdk
from test_gpu_paged import Case, _attend_ref, _i32, _status, _vec

pytestmark = pytest.mark.gpu


def _near(c, out, window=0):
    d = c.q.shape[2]
    want, tol, _, _ = _attend_ref(c.q, c.dk, c.dv, c.pages, c.table, c.lens, c.cu, True, window,
                                  1 / math.sqrt(d))
    return ((out.double() - want).abs() <= tol).all()


# ------------------------------------------------- less work than the bounds

@pytest.mark.parametrize("lens,window", [([50], 0), ([1], 0), ([3, 0, 2], 0), ([262144], 16),
                                         ([262144], 64)], ids=str)
def test_fewer_tokens_than_the_launch(lens, window):
    """Few seen tokens in a call whose bounds admit many: results do not
    depend on what the workspace held, finite or not, nor on an earlier call
    over a longer context."""
    new = [min(x, 1) for x in lens]
    c = Case(lens, new, Hq=2, Hkv=1, n=32768, P=64, cols=4096, seed=21)
    bounds = dict(max_q=1, max_len=262144, total=262144)
    ws = c.workspace(**bounds)
    got = []
    for fill in (0, 0x3F800000, 0x7FC00000, 0x7F800000, -1):
        ws[256:].view(torch.int32).fill_(fill)
        lse = torch.full((c.q.shape[0], 2), 77.0, device="cuda")
        got.append((c.run(window=window, ws=ws, lse=lse, **bounds), lse))
    if window:
        c.run(ws=ws, **bounds)                  # the whole context, and then again
        got.append((c.run(window=window, ws=ws, lse=lse, **bounds), lse))
    assert _status(ws) == (0, 0)
    assert _near(c, got[0][0], window)
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


# --------------------------------------------------------------- NaN queries

@pytest.mark.parametrize("window", [1, 2, 3])
@pytest.mark.parametrize("lens,new", [([500, 900], [140, 1]), ([2000, 20], [4, 1]),
                                      ([40000], [9])], ids=str)
def test_nan_queries_under_short_windows(lens, new, window):
    """A NaN query's row is NaN wherever its few seen tokens lie, its log-sum
    too; the other rows are as before."""
    c = Case(lens, new, seed=22)
    want = c.run(window=window)
    c.q[:, 2] = float("nan")
    lse = torch.zeros(c.q.shape[:2], device="cuda")
    got = c.run(window=window, lse=lse)
    assert torch.isnan(got[:, 2]).all() and torch.isnan(lse[:, 2]).all()
    keep = [h for h in range(8) if h != 2]
    assert torch.equal(got[:, keep], want[:, keep]) and torch.isfinite(lse[:, keep]).all()


# -------------------------------------------------------- pages behind a window

@pytest.mark.parametrize("left", [-1, 1 << 30, "reused"], ids=str)
@pytest.mark.parametrize("lens,new,kw,window", [
    ([700], [129], dict(P=7), 50), ([1500] * 3, [90, 1, 40], dict(P=16, d=64), 200),
    ([9000], [300], dict(P=24), 1000),
    ([1100, 300], [3, 1], dict(P=16), 50), ([1100], [2], dict(P=1, d=64), 7),
    ([40000], [1], dict(P=16, n=32768), 5001), ([40000, 900], [2, 1], dict(P=24, d=64), 3000)], ids=str)
def test_pages_behind_the_window(lens, new, kw, window, left):
    """Pages whose tokens no row sees any more may have left the table, or
    serve others: they are neither looked up nor read."""
    c = Case(lens, new, seed=23, **kw)
    want = c.run(window=window)
    if left == "reused":                        # a page of words that no call may use
        left = (set(range(c.pages.shape[0])) - set(c.table.view(-1).tolist())).pop()
    for b, (L, n) in enumerate(zip(lens, new)):
        gone = max(0, L - n - window + 1) // c.P
        assert gone > 0 or L < 1000
        c.table[b, :gone] = left
    ws = c.workspace()
    assert torch.equal(c.run(window=window, ws=ws), want) and _status(ws) == (0, 0)


# --------------------------------------------------- sizes of weights by atoms

@pytest.mark.parametrize("where", [[5, 900, 39990], [39999], [20000, 20001, 20002, 20003]], ids=str)
def test_heavy_tokens_with_small_values(where):
    """A few tokens have all the weight and values a ten-millionth of the others'
    (whose probabilities are below 2^-50): the weights keep their bits."""
    c = Case([40000], [1], Hq=4, Hkv=2, n=5000, seed=24)
    half = lambda x: x.clamp(-65504, 65504).half().view(torch.int16).to(torch.int32) << 16
    times = lambda w, f: half((w >> 16).to(torch.int16).view(torch.float16).float() * f) | (w & 0x7FFF)
    k, v = c.pages[:, :, :, 0], c.pages[:, :, :, 1]
    good = ((k[..., 0] & 0x7FFF) < 5000)[..., None]           # slots that hold a token
    c.pages[:, :, :, 0] = torch.where(good, times(k, 1e-4), k)
    c.pages[:, :, :, 1] = torch.where(good, times(v, 2e4), v)
    c.q[:] = c.q[:, :1]
    for h in range(2):
        row = c.q[0, 2 * h].double() @ c.dk.double().T / math.sqrt(128)
        atom = int(row.argmax())
        word = half(40.0 / row[atom].float()).item() | atom    # a score of 40: e^40 = 2^57
        for t in where:
            page, off = c.table[0, t // c.P].item(), t % c.P
            c.pages[page, h, off, 0, 0] = word
            c.pages[page, h, off, 1] = times(c.pages[page, h, off, 1], 1e-7)
    c.check()


# -------------------------------------------------- flat long contexts by atoms

def test_flat_attention_over_long_contexts():
    """2.4 million tokens, all of the same weight: sums that cancel keep their
    bits however many tokens an SM adds up.

    Tolerance: an output is a sum of N = 2.4e6 x 16 products of random signs;
    with r its root mean square over rows and dims,
        |out - ref| <= 2^-8 |ref| (bf16) + 1.9e-3 r.
    A product p c is rounded to a multiple of a unit u that is at most
    sum |p c| / 5e8 of its share of S <= 2^15 tokens, that is 16 S mean|pc| / 5e8
    = 1.05e-3 mean|pc|; a rounding's deviation is u / sqrt(12) = 3.0e-4 mean|pc|,
    against sqrt(pi / 2) mean|pc| of the product: 2.4e-4 r after the same sum;
    4096 outputs stay within six deviations: 1.5e-3 r.  The scale of 1e-6 keeps
    scores below 1e-4, known to 1e-4 2^-11, so that even a sum of errors of one
    sign is below 5e-8 / (mean / rms of the sum: 1 / sqrt(N)) = 3e-4 r.  Weights
    as two bf16 parts (2^-17) and fp32 sums add less than 1e-4 r."""
    L, Hkv, Hq, d, n, P = 2400000, 2, 32, 128, 32768, 64
    g = torch.Generator(device="cuda").manual_seed(25)
    n_pages = L // P
    pages = torch.empty(n_pages, Hkv, P, 2, 16, dtype=torch.int32, device="cuda")
    for i in range(0, n_pages, 5000):
        k = min(5000, n_pages - i)
        idx = torch.randint(0, n, (k, Hkv, P, 2, 16), generator=g, device="cuda", dtype=torch.int32)
        c = torch.randn(idx.shape, generator=g, device="cuda").half()
        pages[i:i + k] = (c.view(torch.int16).to(torch.int32) << 16) | idx
    D = torch.randn(2, n, d, generator=g, device="cuda")
    D = (D / D.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    q = (torch.randn(1, Hq, d, generator=g, device="cuda") * 2).to(torch.bfloat16)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    ws = sdk.new_workspace(sdk.sdk_chunk_attn_workspace_bytes(1, 1, Hq, Hkv, d, n, 1, L, L))
    out = sdk.sdk_chunk_attn(q, D[0].contiguous(), D[1].contiguous(), pages, table, _i32([L]),
                             _i32([0, 1]), 1, L, total_len=L, scale=1e-6, workspace=ws)
    assert _status(ws) == (0, 0)
    ref = torch.empty(Hq, d, dtype=torch.float64, device="cuda")
    for h in range(Hkv):
        rec = pages[:, h].reshape(L, 2, 16)
        coef = (rec >> 16).to(torch.int16).view(torch.float16)
        idx = (rec & 0x7FFF).long()
        for r in range(h * 16, h * 16 + 16):
            qd = D[0].double() @ q[0, r].double()
            s = torch.zeros(L, dtype=torch.float64, device="cuda")
            for j in range(16):
                s += coef[:, 0, j].double() * qd[idx[:, 0, j]]
            p = torch.softmax(s * 1e-6, 0)
            w = torch.zeros(n, dtype=torch.float64, device="cuda")
            for j in range(16):
                w.index_add_(0, idx[:, 1, j], p * coef[:, 1, j].double())
            ref[r] = w @ D[1].double()
    err, r = (out[0].double() - ref).abs(), ref.square().mean().sqrt()
    far = err - (2.0 ** -8 * ref.abs() + 1.9e-3 * r)
    assert not (far > 0).any(), "over by %g r at %d places" % (far.max() / r, (far > 0).sum())


# ------------------------------------------------------------- captured plans

def test_plan_replays_on_its_pool():
    """PagedCodeStore.plan captured in a graph: every replay takes pages of
    its own, releases between replays are seen, and a plan without a graph
    goes on where the replays ended."""
    store = sdk.PagedCodeStore(12, 1, 4)
    lens, new, table = _i32([0, 0]), _i32([4, 8]), _i32([[-1] * 8] * 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        store.plan(_i32([0]), _i32([0]), _i32([[-1]]), 1)      # nothing is taken
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = store.plan(lens, new, table, 12)
        lens.copy_(plan.new_lens)
    for k in (1, 2):
        graph.replay()
        assert lens.tolist() == [4 * k, 8 * k] and store.n_free.tolist() == [12 - 3 * k]
        assert plan.n_free.tolist() == [12 - 3 * k]
    held = table[0, :2].tolist() + table[1, :4].tolist()
    assert sorted(held) == list(range(6))
    store.release(table[1, :4].clone())
    assert store.n_free.tolist() == [10]
    lens.copy_(_i32([8, 0]))
    graph.replay()
    assert store.n_free.tolist() == [7] and lens.tolist() == [12, 8]
    plan = store.plan(lens, new, table, 12)
    assert store.n_free.tolist() == [4] and plan.n_free.tolist() == [4]
    held = table[0, :4].tolist() + table[1, :4].tolist()
    assert len(set(held)) == 8


# ------------------------------------------------------------ records of plans

def test_refusals_are_kept_by_the_store():
    """A plan without a workspace records in the store's, until it is read."""
    store = sdk.PagedCodeStore(3, 1, 4)
    table = _i32([[-1] * 4] * 2)
    plan = store.plan(_i32([0, 0]), _i32([4, 9]), table, 13)         # four pages of three
    assert plan.new_lens.tolist() == [4, 0] and plan.cu_new.tolist() == [0, 4, 13]
    assert plan.slot_map.tolist() == [0, 1, 2, 3] + [-1] * 9
    store.plan(_i32([4, 0]), _i32([1, 0]), table, 1)
    assert _status(store.workspace)[0] == 3 and _status(store.workspace)[0] == 0
    ws = sdk.new_workspace(256)
    store.plan(_i32([5, 0]), _i32([0, 9]), table, 9, workspace=ws)
    assert _status(store.workspace)[0] == 0 and _status(ws)[0] == 3


# ------------------------------------------------------------- refused requests

def test_a_refused_request_leaves_the_others():
    """The pool runs out at the second of four requests: the third needs a
    page and is refused too, the fourth needs none and goes on.  The accepted
    ones' slots and rows are those of a step without the others."""
    c = Case([20, 30, 16, 5], [2, 1, 1, 1], P=16, n=100, cols=4, seed=26)
    lens, new = _i32([18, 32, 16, 4]), _i32([2, 20, 3, 1])
    free = _i32([c.pages.shape[0] - 1])
    r = sdk.sdk_block_tables(lens, new, free, _i32([1]), c.table.clone(), 16, 26,
                             n_pages=c.pages.shape[0])
    assert r.new_lens.tolist() == [20, 32, 16, 5] and r.cu_new.tolist() == [0, 2, 22, 25, 26]
    assert r.n_free.tolist() == [1] and r.block_table.tolist() == c.table.tolist()
    assert (r.new_lens != lens + new).tolist() == [False, True, True, False]
    slots = r.slot_map.tolist()
    assert slots[2:25] == [-1] * 23
    at = lambda b, t: c.table[b, t // 16].item() * 16 + t % 16
    assert slots[:2] == [at(0, 18), at(0, 19)] and slots[25] == at(3, 4)
    q = c.q[:1].expand(26, -1, -1).contiguous()
    q[:2], q[25] = c.q[:2], c.q[4]
    out = sdk.sdk_chunk_attn(q, c.dk, c.dv, c.pages, c.table, r.new_lens, r.cu_new, 20, 32)
    want, tol, _, _ = _attend_ref(c.q, c.dk, c.dv, c.pages, c.table, c.lens, c.cu, True, 0,
                                  1 / math.sqrt(128))
    assert ((out[[0, 1, 25]].double() - want[[0, 1, 4]]).abs() <= tol[[0, 1, 4]]).all()


# --------------------------------------------------------------------- workspace

def test_workspace_of_long_contexts():
    """Few rows over long contexts need the form's own buffers (a tenth of an
    fp16 copy of the context, two tenths under loose bounds), and these do."""
    f = sdk.sdk_chunk_attn_workspace_bytes
    fp16 = lambda tokens, Hkv=8, d=128: tokens * Hkv * 2 * d * 2
    assert f(1, 1, 32, 8, 128, 32768, 1, 262144, 262144) < 0.1 * fp16(262144)
    assert f(64, 64, 32, 8, 128, 32768, 1, 32768) < 0.2 * fp16(64 * 32768)
    c = Case([40000, 3000], [1, 1], Hq=8, Hkv=2, n=3000, seed=27)
    c.check()


# ------------------------------------------------------------ outputs in place

@pytest.mark.parametrize("lens,new,kw", [
    ([300, 40], [3, 1], {}), ([2000] * 3, [4, 1, 2], dict(d=64)), ([700, 300], [129, 300], {}),
    ([40000, 50], [2, 1], dict(n=32768))], ids=str)
def test_out_in_place_of_q(lens, new, kw):
    """out may be q itself, whichever form runs."""
    c = Case(lens, new, seed=28, **kw)
    want = c.run()
    q = c.q.clone()
    assert c.run(q=q, out=q) is q and torch.equal(q, want)


def test_out_may_not_lie_partly_on_q():
    c = Case([300], [20], seed=28)
    room = torch.zeros(30, *c.q.shape[1:], dtype=torch.bfloat16, device="cuda")
    room[:20] = c.q
    with pytest.raises(sdk.SdkError, match="SDK_ERR_INVALID_ARG"):
        c.run(q=room[:20], out=room[1:21])
    lse = room.view(torch.float32)[:20].reshape(-1)[:160].view(20, 8)
    with pytest.raises(sdk.SdkError, match="SDK_ERR_INVALID_ARG"):
        c.run(q=room[:20], lse=lse)
    assert torch.equal(room[:20], c.q)


# ------------------------------------------------------ outputs of a plan apart

@pytest.mark.parametrize("given", [(), ("slot_map",), ("cu_new", "n_free_out")])
@pytest.mark.parametrize("B,max_new", [(1, 1), (3, 7), (5, 8), (64, 1001)])
def test_outputs_of_a_plan_lie_apart(B, max_new, given):
    """What is written to one output, from its first to its last byte, does
    not reach another."""
    make = dict(slot_map=lambda: torch.empty(max_new, dtype=torch.int64, device="cuda"),
                cu_new=lambda: _i32([0] * (B + 1)), n_free_out=lambda: _i32([0]))
    r = sdk.sdk_block_tables(_i32([0] * B), _i32([0] * B), _i32([0]), _i32([1]), _i32([[-1]] * B), 4,
                             max_new, **{k: make[k]() for k in given})
    outs = [r.slot_map, r.cu_new, r.new_lens, r.n_free]
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in outs)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    for i, t in enumerate(outs):
        t.fill_(i + 100)
    assert all((t == i + 100).all() for i, t in enumerate(outs))
