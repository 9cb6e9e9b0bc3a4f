"""Block tables and slots from request lengths, and rows into a latent cache,
against the oracle (GB300)."""
import numpy as np
import pytest

from latent_util import HALF_BF16, MODES, torch_dtype, tree_parents, TYPES

import speculative_decoding_verify_kv_gb300 as va
from oracle import latent_oracle as lo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def pool_of(r, ctx, width, blocks):
    table = np.full((len(ctx), width), -1, np.int32)
    ref = np.zeros(blocks, np.int32)
    order, at = r.permutation(blocks), 0
    for i, c in enumerate(ctx):
        h = -(-int(c) // 16)
        table[i, :h] = order[at:at + h]
        at += h
    ref[order[:at]] = 1
    return table, ref


def run_extend(table, ref, ctx, rows, most, mode="chain", kinds=None, parent=None, status=0):
    dev = lambda a, t=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()  # noqa: E731
    t, f = dev(table), dev(ref)
    st = torch.full((1,), status, dtype=torch.int32, device="cuda")
    out = va.verify_attn_pages_extend(va.PagePool(t, f), dev(ctx), dev(rows), most, MODES[mode],
                                      parent=None if parent is None else dev(np.resize(parent, max(most, 1))),
                                      seq_kind=None if kinds is None else dev(kinds, torch.uint8), status=st)
    got = [x.cpu().numpy() for x in (t, f, out["cu_rows"], out["row_seq"], out["position"], out["slot"])]
    return got, st.item()


@pytest.mark.parametrize("mode", ["chain", "tree", "mixed"])
@pytest.mark.parametrize("seqs,most_rows,most_ctx,spare,pad", [
    (1, 1, 0, 1, 0), (1, 32, 40, 9, 3), (7, 5, 100, 3, 0), (40, 1, 2000, 300, 5), (300, 8, 500, 900, 17),
    (33, 32, 3000, 20000, 1), (1500, 3, 60, 400, 2), (2500, 2, 40, 100, 0),
])
def test_extend(mode, seqs, most_rows, most_ctx, spare, pad):
    r = np.random.default_rng(seqs * 7 + most_rows)
    ctx = r.integers(0, most_ctx + 1, seqs)
    rows = r.integers(0, most_rows + 1, seqs)
    rows[0] = most_rows
    kinds = np.array([1 if mode == "tree" or (mode == "mixed" and i % 3) else 0 for i in range(seqs)])
    width = (most_ctx + most_rows) // 16 + 2
    blocks = int((-(-ctx // 16)).sum() + (-(-(ctx + rows) // 16)).sum() - (-(-ctx // 16)).sum()) + spare
    table, ref = pool_of(r, ctx, width, blocks)
    parent = tree_parents(r, rows, kinds)
    most = int(rows.sum()) + pad
    want = lo.extend(table, ref, ctx, rows, most, kinds, parent)
    assert want[6] == 0
    got, st = run_extend(table, ref, ctx, rows, most, mode, kinds, parent)
    assert st == 0
    for a, b in zip(got, want[:6]):
        assert np.array_equal(a, b)


def test_extend_segments_and_held_pages():
    """Long segments; entries behind a window are gone, some ahead are held already."""
    r = np.random.default_rng(5)
    ctx, rows = np.array([17, 0, 4000, 31, 64]), np.array([5000, 777, 1, 1, 0])
    table, ref = pool_of(r, ctx, 400, 1200)
    ref[table[2, :200]] = 0
    table[2, :200] = -1
    page = int(np.flatnonzero(ref == 0)[-1])
    table[3, 2], ref[page] = page, 1
    most = int(rows.sum())
    want = lo.extend(table, ref, ctx, rows, most)
    got, st = run_extend(table, ref, ctx, rows, most)
    assert st == 0 == want[6] and all(np.array_equal(a, b) for a, b in zip(got, want[:6]))


@pytest.mark.parametrize("blocks", [64, 40000])
@pytest.mark.parametrize("what", ["rows", "most", "ctx", "negative", "shared", "missing", "outside", "parent", "pages",
                                  "count", "tree", "status"])
def test_extend_findings(blocks, what):
    """Nothing changes, the offsets are 0 and the rows -1 (one CTA, and a cluster)."""
    r = np.random.default_rng(1)
    ctx, rows, kinds = np.array([20, 33, 16]), np.array([3, 4, 2]), np.array([0, 1, 1])
    table, ref = pool_of(r, ctx, 5, blocks)
    parent, most, status, bits = tree_parents(r, rows, kinds), 9, 0, None
    if what == "rows":
        rows[1] = -2
    elif what == "most":
        most = 8
    elif what == "ctx":
        ctx[0] = 79
    elif what == "negative":
        ctx[2] = -1
    elif what == "shared":
        ref[table[0, 1]] = 2
    elif what == "missing":
        table[1, 2] = -1
    elif what == "outside":
        table[1, 2] = blocks
    elif what == "parent":
        parent[4] = 1
    elif what == "pages":
        ref[ref == 0] = 1
    elif what == "count":
        ref[np.flatnonzero(ref == 0)[-1]] = -1
    elif what == "tree":
        ctx[2], rows[2], most = 0, 33, 60
        parent = np.zeros(60, np.int32)
    else:
        status = bits = 0x40
    want = lo.extend(table, ref, ctx, rows, most, kinds, parent)
    got, st = run_extend(table, ref, ctx, rows, most, "mixed", kinds, parent, status)
    assert st == (bits or want[6]) and st != 0
    assert np.array_equal(got[0], table) and np.array_equal(got[1], ref)
    assert not got[2].any() and all((x == -1).all() for x in got[3:])


def test_extend_captured():
    """A captured step, replayed as its request grows."""
    table, ref = torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), torch.zeros(16, dtype=torch.int32, device="cuda")
    ctx, rows = torch.tensor([0, 0], dtype=torch.int32, device="cuda"), torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    call = va.ExtendCall(va.PagePool(table, ref), ctx, rows, 16)
    call()
    table.fill_(-1)
    ref.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
        ctx.add_(rows)
    t, f, c = table.cpu().numpy(), ref.cpu().numpy(), np.array([0, 0])
    for _ in range(5):
        graph.replay()
        t, f, *rest, bad = lo.extend(t, f, c, np.array([5, 9]), 16)
        assert bad == 0
        for a, b in zip([table, ref, out["cu_rows"], out["row_seq"], out["position"], out["slot"]], [t, f, *rest]):
            assert np.array_equal(a.cpu().numpy(), b)
        c = c + [5, 9]


def append_case(kind, rows, heads, latent, pad, offset, seed):
    dt, width = torch_dtype(kind), latent + 64
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(rows, width + pad, generator=g).mul_(2).to(dt)
    slots, positions = rows + 9, 50
    angle = torch.arange(positions)[:, None] * 10000.0 ** (-torch.arange(32) / 32.0)
    qw = torch.randn(rows, heads, 64 + pad, generator=g).to(dt)
    return dict(kv=wide[:, offset:offset + width], cache=torch.randn(slots, width, generator=g).to(dt),
                slot=torch.randperm(slots, generator=g)[:rows],
                position=torch.randint(0, positions, (rows,), generator=g, dtype=torch.int32),
                rope=torch.cat([angle.cos(), angle.sin()], 1).float(),
                weight=(1 + 0.1 * torch.randn(latent, generator=g)).to(dt),
                q_rope=qw[..., offset:offset + 64], q=torch.randn(rows, heads, width, generator=g).to(dt))


def gpu_strided(t):
    """The tensor on the GPU with the strides it has here."""
    if t.is_contiguous():
        return t.cuda()
    base = t._base.cuda()
    return base.as_strided(t.shape, t.stride(), t.storage_offset())


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,pad,offset,norm", [
    (1, 1, 0, 0, True), (1, 16, 0, 0, True), (5, 128, 0, 0, False), (77, 5, 8, 8, True), (9, 3, 7, 3, True),
    (3, 0, 0, 0, True), (400, 40, 1, 0, False), (2, 256, 24, 16, True),
])
def test_append(kind, latent, interleaved, rows, heads, pad, offset, norm):
    c = append_case(kind, rows, heads, latent, pad, offset, rows + heads)
    gpu = {k: gpu_strided(v) for k, v in c.items()}
    kv = va.LatentKV(TYPES[kind], latent, 64, gpu["cache"], capacity=gpu["cache"].shape[0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = va.LatentRows(gpu["kv"], gpu["position"], gpu["slot"], gpu["rope"], norm_weight=gpu["weight"] if norm else None,
                        norm_eps=1e-5, interleaved=interleaved, q_rope=gpu["q_rope"] if heads else None,
                        q=gpu["q"] if heads else None)
    va.verify_attn_latent_append(kv, new, status=status)
    assert status.item() == 0
    d = {k: v.double().numpy() if v.is_floating_point() else v.numpy() for k, v in c.items()}
    cache, q = lo.append(d["cache"], d["kv"], d["position"], d["slot"], d["rope"], d["weight"] if norm else None, 1e-5,
                         interleaved, d["q_rope"], d["q"])
    # One rounding to the type; before it a product or two and, for the norm, a
    # mean of up to 512 squares (a random walk of roundings, and 2^-24 for each of
    # a handful of operations): 2e-6 of a value, and of the pair's size in a turn.
    step = HALF_BF16 if kind == "bf16" else 2.0 ** -24
    for got, want, big in ((gpu["cache"], cache, 12.0), (gpu["q"], q, 6.0)):
        got = got.double().cpu().numpy()
        assert (np.abs(got - want) <= step * np.abs(want) * (1 + 1e-6) + 2e-6 * (np.abs(want) + big / 10)).all()
    left = np.setdiff1d(np.arange(len(cache)), d["slot"])
    assert torch.equal(gpu["cache"].cpu()[left], c["cache"][left])
    assert torch.equal(gpu["q"].cpu()[..., :latent], c["q"][..., :latent])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_append_skips(kind):
    """Padding rows, rows without a slot, bad slots and positions."""
    c = append_case(kind, 6, 4, 256, 0, 0, 3)
    c["slot"][1], c["slot"][2], c["slot"][5] = -1, 10 ** 12, -7
    c["position"][3], c["position"][4] = -1, 50
    gpu = {k: v.cuda() for k, v in c.items()}
    kv = va.LatentKV(TYPES[kind], 256, 64, gpu["cache"], capacity=gpu["cache"].shape[0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    va.verify_attn_latent_append(kv, va.LatentRows(gpu["kv"], gpu["position"], gpu["slot"], gpu["rope"],
                                                   q_rope=gpu["q_rope"], q=gpu["q"]), status=status)
    assert status.item() == va.DEV_BAD_BLOCK | va.DEV_CTX_OVERFLOW
    same = (gpu["cache"].cpu() == c["cache"]).all(1)
    assert same.sum() == len(same) - 1 and not same[c["slot"][0]]
    turned = (gpu["q"].cpu() != c["q"]).flatten(1).any(1)
    assert turned.tolist() == [True, True, False, False, False, False]


def test_append_queries_in_place():
    c = append_case("bf16", 7, 6, 512, 0, 0, 8)
    a, b = c["q"].cuda(), c["q"].cuda()
    cache = c["cache"].cuda()
    kv = va.LatentKV(va.BF16, 512, 64, cache, capacity=cache.shape[0])
    args = [c[k].cuda() for k in ("kv", "position", "slot", "rope")]
    va.verify_attn_latent_append(kv, va.LatentRows(*args, q_rope=a[..., 512:].clone(), q=a))
    va.verify_attn_latent_append(kv, va.LatentRows(*args, q_rope=b[..., 512:], q=b))
    assert torch.equal(a, b)
