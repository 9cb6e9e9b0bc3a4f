"""Pages of a paged cache on the GPU against the oracle: whole numbers and
copied bytes, equal."""
import numpy as np
import pytest

import oracle.step_oracle as so

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verify_kv_gb300 as va  # noqa: E402

BITS = {"rows": va.DEV_BAD_ROWS, "overflow": va.DEV_CTX_OVERFLOW, "block": va.DEV_BAD_BLOCK,
        "pages": va.DEV_NO_PAGES}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def random_pool(seed, seqs, width, blocks, shared=0.3, holes=0.1):
    """A consistent pool: rows of random length, some first pages shared."""
    g = np.random.default_rng(seed)
    perm = g.permutation(blocks)
    table = np.full((seqs, width), -1, np.int32)
    at, lens = 0, []
    for s in range(seqs):
        n = int(g.integers(0, width + 1))
        n = min(n, (blocks - at))
        share = 0
        if s and g.random() < shared:
            o = int(g.integers(0, s))
            share = min(n, int((table[o] >= 0).sum()), lens[o])
            table[s, :share] = table[o, :share]
        table[s, share:n] = perm[at:at + n - share]
        at += n - share
        lens.append(n)
        if g.random() < holes and n > 2:
            table[s, 0:n // 2] = -1
    ref = np.zeros(blocks, np.int32)
    np.add.at(ref, table[table >= 0], 1)
    return table, ref, lens


def fork(table, ref, src, dst, length, pages, status=0):
    t, r = dev(table), dev(ref)
    st = torch.tensor([status], dtype=torch.int32, device="cuda")
    copies = torch.full((len(src), 2), -9, dtype=torch.int32, device="cuda")
    copies, n = va.verify_attn_pages_fork(va.PagePool(t, r), dev(src), dev(dst), dev(length), dev(pages),
                                          copies=copies, status=st)
    torch.cuda.synchronize()
    return t.cpu().numpy(), r.cpu().numpy(), copies.cpu().numpy(), int(n.item()), int(st.item())


def check_fork(table, ref, src, dst, length, pages):
    t, r, copies, bad = so.pages_fork(table, ref, src, dst, length, pages)
    gt, gr, gc, gn, gs = fork(table, ref, src, dst, length, pages)
    bits = 0
    for b in bad:
        bits |= BITS[b]
    assert gs == bits, (hex(gs), bad)
    assert np.array_equal(gt, t) and np.array_equal(gr, r)
    assert gn == len(copies) and gc[:gn].tolist() == [list(c) for c in copies]
    assert (gc[gn:] == -9).all()
    return bad


@pytest.mark.parametrize("seqs,width,blocks", [(2, 1, 3), (4, 5, 40), (40, 33, 900), (300, 70, 9000),
                                               (16, 600, 33000)])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_fork_and_grow(seqs, width, blocks, seed):
    g = np.random.default_rng(seed + 100 * seqs)
    table, ref, lens = random_pool(seed, seqs, width, blocks)
    order = g.permutation(seqs)
    srcs, dsts = order[:seqs // 2], order[seqs // 2:]
    src, dst, length, pages = [], [], [], []
    for d in dsts:
        if g.random() < 0.4:  # grow
            n = int(g.integers(0, 16 * lens[d] + 1))
            src.append(d), dst.append(d), length.append(n)
            pages.append(int(g.integers(-(-n // 16), width + 1)))
        else:
            s = int(g.choice(srcs))
            n = int(g.integers(0, 16 * lens[s] + 1))
            if n % 16 and table[s, n // 16] < 0:
                n -= n % 16
            src.append(s), dst.append(d), length.append(n)
            pages.append(int(g.integers(-(-n // 16), min(width, -(-n // 16) + 3) + 1)))
    check_fork(table, ref, src, dst, length, pages)


def test_fork_errors_change_nothing():
    table = np.array([[5, 2, 7, -1], [-1] * 4, [3, -1, -1, -1], [-1] * 4], np.int32)
    ref = np.array([0, 0, 1, 1, 0, 1, 0, 1], np.int32)
    ok = ([0], [1], [33], [4])
    assert not check_fork(table, ref, *ok)
    for bad in [([0], [4], [1], [1]), ([-1], [1], [1], [1]), ([0], [1], [33], [2]), ([0], [1], [-1], [1]),
                ([0], [1], [65], [5]), ([0], [1], [0], [-1]), ([0, 2], [1, 1], [3, 3], [1, 1]),
                ([0, 1], [1, 3], [3, 0], [1, 1]), ([1], [2], [3], [1]), ([0], [1], [60], [4]),
                ([0, 2, 0], [1, 2, 3], [48, 16, 48], [4, 4, 4]), ([0, 0], [0, 1], [48, 33], [4, 4])]:
        assert check_fork(table, ref, *bad), bad
    for entry in (8, -2, 0, 4):  # outside the pool, or a page that is free
        t = table.copy()
        t[0, 1] = entry
        assert check_fork(t, ref, *ok) == {"block"}
    r = ref.copy()
    r[6] = -1
    assert check_fork(table, r, *ok) == {"block"}
    # A status word that already holds a finding: nothing is done.
    got = fork(table, ref, *ok, status=va.DEV_TIMEOUT)
    assert np.array_equal(got[0], table) and np.array_equal(got[1], ref) and got[3] == 0 and got[4] == va.DEV_TIMEOUT


def test_fork_takes_the_last_free_page_and_not_one_more():
    table = np.array([[0, -1], [-1, -1]], np.int32)
    assert not check_fork(table, np.array([1, 0, 0], np.int32), [0], [1], [7], [2])
    assert check_fork(table, np.array([1, 0], np.int32), [0], [1], [7], [2]) == {"pages"}


def test_no_commands():
    table, ref, _ = random_pool(3, 4, 5, 40)
    gt, gr, _, n, st = fork(table, ref, [], [], [], [])
    assert np.array_equal(gt, table) and np.array_equal(gr, ref) and n == 0 and st == 0


def free(table, ref, seq, first, last, status=0):
    t, r = dev(table), dev(ref)
    st = torch.tensor([status], dtype=torch.int32, device="cuda")
    va.verify_attn_pages_free(va.PagePool(t, r), dev(seq), dev(first), dev(last), status=st)
    torch.cuda.synchronize()
    return t.cpu().numpy(), r.cpu().numpy(), int(st.item())


@pytest.mark.parametrize("seqs,width,blocks", [(2, 1, 3), (4, 5, 40), (300, 70, 9000), (16, 600, 33000)])
def test_free(seqs, width, blocks):
    g = np.random.default_rng(seqs)
    table, ref, _ = random_pool(seqs, seqs, width, blocks, shared=0.6)
    n = seqs * 2  # some sequences more than once, ranges that overlap
    seq = g.integers(0, seqs, n)
    ends = np.sort(g.integers(0, width + 1, (n, 2)), axis=1)
    t, r, bad = so.pages_free(table, ref, seq, ends[:, 0], ends[:, 1])
    gt, gr, gs = free(table, ref, seq, ends[:, 0], ends[:, 1])
    assert not bad and gs == 0 and np.array_equal(gt, t) and np.array_equal(gr, r)


def test_free_errors_change_nothing():
    table = np.array([[5, 2, 7, -1], [5, 2, -1, -1]], np.int32)
    ref = np.array([0, 0, 2, 0, 0, 2, 0, 1], np.int32)
    for seq, a, b, bit in [([0, 2], [0, 0], [1, 1], "rows"), ([0, -1], [0, 0], [1, 1], "rows"),
                           ([0], [2], [1], "overflow"), ([0], [0], [5], "overflow"), ([0], [-1], [1], "overflow")]:
        gt, gr, gs = free(table, ref, seq, a, b)
        assert gs == BITS[bit] and np.array_equal(gt, table) and np.array_equal(gr, ref)
    t = table.copy()
    t[1, 1] = 99
    gt, gr, gs = free(t, ref, [0, 1], [0, 0], [4, 4])
    assert gs == va.DEV_BAD_BLOCK and np.array_equal(gt, t) and np.array_equal(gr, ref)
    # More entries than references: the count stays at 0, and is reported.
    r = ref.copy()
    r[5] = 1
    gt, gr, gs = free(table, r, [0, 1], [0, 0], [4, 4])
    assert gs == va.DEV_BAD_BLOCK and (gt == -1).all() and (gr == 0).all()


def compact(table, ref, status=0):
    t, r = dev(table), dev(ref)
    st = torch.tensor([status], dtype=torch.int32, device="cuda")
    copies = torch.full((len(ref) // 2, 2), -9, dtype=torch.int32, device="cuda")
    copies, n, live = va.verify_attn_pages_compact(va.PagePool(t, r), copies=copies, status=st)
    torch.cuda.synchronize()
    return t.cpu().numpy(), r.cpu().numpy(), copies.cpu().numpy(), int(n.item()), int(live.item()), int(st.item())


def check_compact(table, ref):
    t, r, copies, live, bad = so.pages_compact(table, ref)
    gt, gr, gc, gn, gl, gs = compact(table, ref)
    assert gs == (va.DEV_BAD_BLOCK if bad else 0)
    assert np.array_equal(gt, t) and np.array_equal(gr, r)
    assert gn == len(copies) and gc[:gn].tolist() == [list(c) for c in copies] and (gc[gn:] == -9).all()
    if not bad:
        assert gl == live


@pytest.mark.parametrize("seqs,width,blocks", [(1, 1, 1), (2, 1, 3), (4, 5, 40), (7, 9, 31), (7, 9, 32),
                                               (300, 70, 9000), (16, 600, 33000), (3, 40, 8192 * 4 + 5)])
@pytest.mark.parametrize("seed", [0, 1])
def test_compact(seqs, width, blocks, seed):
    table, ref, _ = random_pool(seed + 7, seqs, width, blocks, shared=0.5)
    check_compact(table, ref)


def test_compact_of_full_empty_and_packed_pools():
    check_compact(np.full((2, 3), -1, np.int32), np.zeros(70, np.int32))
    check_compact(np.arange(64, dtype=np.int32).reshape(2, 32), np.ones(64, np.int32))
    check_compact(np.arange(64, dtype=np.int32).reshape(2, 32), np.r_[np.ones(64), np.zeros(64)].astype(np.int32))
    # The pages in use all at the end.
    check_compact(np.arange(64, 128, dtype=np.int32).reshape(2, 32), np.r_[np.zeros(64), np.ones(64)].astype(np.int32))
    check_compact(np.array([[0, 5]], np.int32), np.array([1, 0, 0, 0, 0, 0], np.int32))  # a free page in the table
    got = compact(np.array([[5]], np.int32), np.array([0, 0, 0, 0, 0, 1], np.int32), status=va.DEV_BAD_ROWS)
    assert got[0].tolist() == [[5]] and got[3] == 0 and got[5] == va.DEV_BAD_ROWS


@pytest.mark.parametrize("page_bytes", [16, 48, 2176, 4352, 16384, 17408, 32768])
@pytest.mark.parametrize("pools", [1, 5, 64, 67])
def test_copy(page_bytes, pools):
    blocks, n = 60, 13
    g = torch.Generator().manual_seed(page_bytes + pools)
    host = [torch.randint(0, 255, (blocks, page_bytes), generator=g, dtype=torch.uint8) for _ in range(pools)]
    order = torch.randperm(blocks, generator=g).tolist()
    pairs = [[order[i], order[30 + i]] for i in range(n)]
    want = [h.clone() for h in host]
    for h in want:
        for a, b in pairs:
            h[b] = h[a]
    got = [h.cuda() for h in host]
    copies = dev(pairs + [[1, 2]] * 3)  # entries past the count are not looked at
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    va.verify_attn_pages_copy(got, copies, dev([n]), status=st)
    assert int(st.item()) == 0
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), b)


def test_copy_passes_over_bad_pairs_and_failed_plans():
    pool = torch.arange(10 * 4, dtype=torch.int32).reshape(10, 4).cuda()
    ref = pool.clone()
    st = torch.tensor([va.DEV_NO_PAGES], dtype=torch.int32, device="cuda")
    va.verify_attn_pages_copy([pool], dev([[0, 1]]), dev([1]), status=st)
    assert torch.equal(pool, ref) and int(st.item()) == va.DEV_NO_PAGES
    st.zero_()
    va.verify_attn_pages_copy([pool], dev([[0, 1], [10, 2], [3, -1], [4, 5]]), dev([4]), status=st)
    ref[1], ref[5] = ref[0], ref[4]
    assert torch.equal(pool, ref) and int(st.item()) == va.DEV_BAD_COPY
    st.zero_()
    va.verify_attn_pages_copy([pool], dev([[6, 7]]), dev([5]), status=st)  # a count past the list's end
    ref[7] = ref[6]
    assert torch.equal(pool, ref) and int(st.item()) == va.DEV_BAD_COPY
    st.zero_()
    va.verify_attn_pages_copy([pool], dev([[6, 8]]), dev([-3]), status=st)
    assert torch.equal(pool, ref) and int(st.item()) == 0


def test_copy_of_offsets_past_32_bits():
    """A pool of 4.5 GB: the pages at its two ends."""
    blocks = 140000
    pool = torch.zeros(blocks, 8192, dtype=torch.int32, device="cuda")
    pool[blocks - 1] = torch.arange(8192, dtype=torch.int32, device="cuda")
    pool[3] = 7
    va.verify_attn_pages_copy([pool], dev([[blocks - 1, 0], [3, blocks - 2]]), dev([2]))
    assert torch.equal(pool[0], pool[blocks - 1]) and (pool[blocks - 2] == 7).all()
    assert (pool[1:3] == 0).all() and (pool[blocks - 3] == 0).all()


def test_a_captured_fork_and_copy_replays():
    table, ref, _ = random_pool(11, 8, 6, 200)
    t, r = dev(table), dev(ref)
    t0, r0 = t.clone(), r.clone()
    pool = torch.randint(0, 1000, (200, 64), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    live = np.where((table >= 0).sum(1) > 1)[0]
    src, dst = int(live[0]), int(live[-1])
    n = int((table[src] >= 0).sum())
    first = int(np.where(table[src] >= 0)[0][-1])
    args = [dev([src]), dev([dst]), dev([first * 16 + 5]), dev([first + 1])]
    plan = va.ForkCall(va.PagePool(t, r), *args, status=st)
    copy = va.PageCopyCall([pool], plan._out[0], plan._out[1], status=st)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        plan()
        copy()
    torch.cuda.synchronize()
    want = so.pages_fork(table, ref, [src], [dst], [first * 16 + 5], [first + 1])
    with torch.cuda.graph(g):
        plan()
        copy()
    for _ in range(2):
        t.copy_(t0), r.copy_(r0)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(r.cpu().numpy(), want[1])
        (a, b), = want[2]
        assert torch.equal(pool[a], pool[b]) and int(st.item()) == 0
    assert n > 1


def test_buffers_of_a_call_on_another_stream_outlive_it():
    """A call that is dropped while its stream has yet to run it: its
    workspace, outputs and arguments are not handed out again before."""
    pool = va.PagePool(torch.full((2, 64), -1, dtype=torch.int32, device="cuda"),
                       torch.zeros(1 << 16, dtype=torch.int32, device="cuda"))
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    side = torch.cuda.Stream()
    call = va.ForkCall(pool, i32(0), i32(0), i32(0), i32(40))
    held = {t.data_ptr() for t in call._own + call._keep[1:5]}  # workspace, outputs, and the commands made for it
    assert len(held) == 7
    torch.full((1,), 255, dtype=torch.uint8, device="cuda")  # (the fill below is loaded by now)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000_000)  # a second
    call(side)
    sizes = [t.numel() * t.element_size() for t in call._own + call._keep[1:5]]
    del call
    again = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    assert not side.query()  # still asleep
    assert not held & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert pool.block_table[0].tolist() == list(range(40)) + [-1] * 24
