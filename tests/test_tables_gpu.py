"""ftd_build_tables against a stack of pages moved one by one on the host: growth, shrinking, beginnings and
ends in one call, too few pages, updates in place, contiguous contexts, capacities, bad entries and lengths."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


def pages(n, ps):
    return -(-max(int(n), 0) // ps)


def plain(old, new, table, free, n_free, ps, lmax, num_pages):
    """The definition, one page at a time.  Returns served, table, free, n_free, tokens as (slot, position)."""
    table, stack = table.copy(), list(free[:n_free])
    served = list(new)
    fits = [o <= lmax and n <= lmax for o, n in zip(old, new)]
    for b, (o, n) in enumerate(zip(old, new)):
        if fits[b]:
            stack += [table[b, i] for i in range(pages(n, ps), pages(o, ps))]
    asked, room, n_stack = 0, [], len(stack)
    for b, (o, n) in enumerate(zip(old, new)):
        k = max(0, pages(n, ps) - pages(o, ps)) if fits[b] else 0
        asked += k
        room.append(fits[b] and (k == 0 or asked <= n_stack))
        if not room[b]:
            served[b] = o
        else:
            for i in range(pages(o, ps), pages(n, ps)):
                table[b, i] = stack.pop()
    out = free.copy()
    out[:len(stack)] = stack
    tokens = [(b, j) for b in range(len(old)) if room[b] for j in range(max(int(old[b]), 0), max(int(new[b]), 0))]
    return np.array(served), table, out, len(stack), tokens


def layout(old, ps, lmax, num_pages, rng):
    """A shuffled pool: tables of the slots' pages and the free list of the others."""
    order = rng.permutation(num_pages).astype(np.int32)
    table = np.full((len(old), -(-lmax // ps)), -7, np.int32)
    k = 0
    for b, o in enumerate(old):
        n = pages(o, ps) if o <= lmax else 0
        table[b, :n] = order[k:k + n]
        k += n
    free = np.full(num_pages, -9, np.int32)
    free[:num_pages - k] = order[k:]
    return table, free, num_pages - k


def make(B, lmax, ps=0, num_pages=0):
    return ftd.DecodeStep(B, 2, 1, 64, lmax, "bf16", "bf16", page_size=ps, num_pages=num_pages)


def check(old, new, ps, lmax, num_pages, cap=None, inplace="", seed=1, status=ftd.FTD_OK, shift=0):
    import torch
    rng = np.random.default_rng(seed)
    B = len(old)
    table, free, n_free = layout(old, ps, lmax, num_pages, rng)
    want = plain(old, new, table, free, n_free, ps, lmax, num_pages)
    total = len(want[4])
    cap = total + 5 if cap is None else cap
    step = make(B, lmax, ps, num_pages)
    t_old, t_new = dev(np.array(old, np.int32)), dev(np.array(new, np.int32))
    t_table, t_free, t_n = dev(table), dev(free), dev(np.array([n_free], np.int32))
    served = t_old if "old" in inplace else t_new if "new" in inplace else torch.full_like(t_old, 99)
    n_out = t_n if "n" in inplace.split("+") else torch.full_like(t_n, 99)
    offsets = torch.full((B + 1,), 99, dtype=torch.int32, device="cuda")
    slots, positions = (torch.full((cap + 8,), 99, dtype=torch.int32, device="cuda")[shift:shift + cap] for _ in range(2))
    before = ftd.ftd_kernel_launches()
    step.tables(t_old, t_new, served, block_table=t_table, free_pages=t_free, n_free=t_n,
                n_free_out=None if n_out is t_n else n_out, offsets=offsets, slots=slots, positions=positions)
    torch.cuda.synchronize()
    assert ftd.ftd_kernel_launches() == before + 1
    assert step.get_error() == status
    assert served.tolist() == want[0].tolist()
    assert np.array_equal(t_table.cpu().numpy(), want[1])
    assert np.array_equal(t_free.cpu().numpy(), want[2])
    assert n_out.tolist() == [want[3]]
    count = np.zeros(B, np.int64)
    for b, _ in want[4]:
        count[b] += 1
    assert offsets.tolist() == [0] + np.cumsum(count).tolist()
    m = min(total, cap)
    assert positions.tolist() == [j for _, j in want[4]][:m] + [0] * (cap - m)
    assert slots.tolist() == [int(want[1][b, j // ps]) * ps + j % ps for b, j in want[4]][:m] + [-1] * (cap - m)
    step.close()


def lengths(kind, B, hi, seed):
    rng = np.random.default_rng(seed)
    a, b = rng.integers(0, hi + 1, B), rng.integers(0, hi + 1, B)
    if kind == "step":
        return np.minimum(a, hi - 1), np.minimum(a, hi - 1) + 1
    if kind == "admit":
        return np.where(rng.random(B) < 0.5, 0, -1), b
    if kind == "end":
        return a, np.where(rng.random(B) < 0.5, -1, 0)
    a, b = np.where(rng.random(B) < 0.3, -3, a), np.where(rng.random(B) < 0.3, -1, b)
    return a, np.where(rng.random(B) < 0.2, a, b)  # some stay as they are


@pytest.mark.parametrize("B,hi,ps", [(1, 1, 128), (1, 700, 128), (3, 300, 256), (33, 1500, 128), (257, 513, 256), (1024, 260, 128)])
@pytest.mark.parametrize("kind", ["step", "admit", "end", "churn"])
def test_lengths(B, hi, ps, kind):
    old, new = lengths(kind, B, hi, B + hi)
    lmax = -(-hi // 16) * 16
    need = sum(pages(max(o, n), ps) for o, n in zip(old, new))
    check(old.tolist(), new.tolist(), ps, lmax, need + 3)


@pytest.mark.parametrize("inplace", ["n", "old", "new", "n+old", "n+new"])
def test_in_place(inplace):
    old, new = lengths("churn", 40, 900, 5)
    check(old.tolist(), new.tolist(), 128, 912, 320, inplace=inplace)


def test_page_ends():
    """Lengths at, before and behind the ends of pages, and of the table."""
    ls = [0, 1, 127, 128, 129, 255, 256, 257, 400]
    old, new = [a for a in ls for _ in ls], [b for _ in ls for b in ls]
    check(old, new, 128, 400, sum(4 for _ in old))


@pytest.mark.parametrize("spare", [0, 1, 2, 5, 9])
def test_too_few_pages(spare):
    """Slots are served in order; once one waits, so do the later ones that ask, but not those that do not."""
    old = [128, 0, 256, 60, 300, -1, 10, 512]
    new = [129, 600, 100, 61, 301, 128, 129, 0]  # asks 1, 5, gives 1, 0, 0, 1, 1, gives 4
    held = sum(pages(o, 128) for o in old)
    check(old, new, 128, 640, held + spare)
    # nothing comes back: the first asks for more than there is
    check([0, 0, 5], [640, 128, 6], 128, 640, 1 + spare)


def test_lengths_too_long():
    check([10, 700, 0, 20], [20, 100, 641, 21], 128, 640, 9, status=ftd.FTD_ERR_SEQ_OVERFLOW)


@pytest.mark.parametrize("cap,shift", [(0, 0), (1, 1), (50, 0), (50, 3), (51, 0), (64, 2)])
def test_capacity(cap, shift):
    """Maps shorter than the new tokens (an error) and longer, on and off 16-byte boundaries."""
    old, new = [3, 0, 127], [20, 30, 131]  # 17 + 30 + 4 = 51
    check(old, new, 128, 256, 8, cap=cap, shift=shift, status=ftd.FTD_ERR_SEQ_OVERFLOW if 0 < cap < 51 else ftd.FTD_OK)


def test_contiguous():
    import torch
    B, lmax = 5, 96
    old, new = np.array([0, 96, -1, 17, 40], np.int32), np.array([96, 0, 5, 18, 40], np.int32)
    step = make(B, lmax)
    served, offsets = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(120, dtype=torch.int32, device="cuda")
    step.tables(dev(old), dev(new), served, offsets=offsets, slots=slots)
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    want = [b * lmax + j for b in range(B) for j in range(max(old[b], 0), max(new[b], 0))]
    assert served.tolist() == new.tolist() and offsets.tolist() == [0, 96, 96, 101, 102, 102]
    assert slots.tolist() == want + [-1] * (120 - len(want))
    step.tables(dev(old), dev(new), served, offsets=offsets)  # no maps
    step.tables(dev(old), dev(new), served)
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    step.close()


def test_bad_entries():
    """Pages outside the pool raise the error; their tokens get no slot, other slots theirs."""
    import torch
    step = make(3, 512, 128, 8)
    for what in ("free", "held", "back", "n_free", "double"):
        table = np.full((3, 4), -1, np.int32)
        table[0, 0], table[1, :2], table[2, 0] = 0, (1, 2), 3
        free = np.array([4, 5, 6, 7, -1, -1, -1, -1], np.int32)
        n_free = 4
        old, new = np.array([100, 200, 100], np.int32), np.array([140, 100, 101], np.int32)
        if what == "free":
            free[3], old[1] = 8, 100  # nothing comes back: the top of the list is handed out
            table[1, 1] = -1
        elif what == "held":
            table[2, 0] = -5
        elif what == "back":
            table[1, 1] = 1 << 30  # comes back and goes to slot 0
        elif what == "n_free":
            n_free = 9
        else:
            n_free, old[0], new[0] = 8, 10, 10  # a page comes back to a full list
        served, n_out = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        slots = torch.zeros(64, dtype=torch.int32, device="cuda")
        step.tables(dev(old), dev(new), served, block_table=dev(table), free_pages=dev(free),
                    n_free=dev(np.array([n_free], np.int32)), n_free_out=n_out, slots=slots)
        torch.cuda.synchronize()
        assert step.get_error() == ftd.FTD_ERR_BAD_PAGE, what
        assert 0 <= int(n_out) <= 8
        s = slots.tolist()
        grown = int(new[0] - old[0])
        if what in ("free", "back"):
            assert s[:28] == list(range(100, 128)) and s[28:40] == [-1] * 12 and s[40] == 3 * 128 + 100
        elif what == "held":
            assert s[grown] == -1
        else:
            assert s[grown] == 3 * 128 + 100
    step.close()


def test_graph_streams_and_repeats():
    """Captured, replayed with the lists updated in place, on a stream of its own; two graphs of one context in turn."""
    import torch
    B, ps, lmax, num = 37, 128, 1024, 200
    rng = np.random.default_rng(3)
    old = rng.integers(0, 400, B).astype(np.int32)
    table, free, n_free = layout(old, ps, lmax, num, rng)
    step = make(B, lmax, ps, num)
    lens, new = dev(old), dev(old)
    t_table, t_free, t_n = dev(table), dev(free), dev(np.array([n_free], np.int32))
    slots = [torch.zeros(3 * B, dtype=torch.int32, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            new.copy_(lens + 2 + k)
            step.tables(lens, new, lens, block_table=t_table, free_pages=t_free, n_free=t_n, slots=slots[k])
        graphs.append(g)
    cur = old.copy()
    for i in range(24):
        k = i % 2
        graphs[k].replay()
        nxt = cur + 2 + k
        w = plain(cur.tolist(), nxt.tolist(), table, free, n_free, ps, lmax, num)
        cur, table, free, n_free = w[0].astype(np.int32), w[1], w[2], w[3]
        torch.cuda.synchronize()
        assert lens.tolist() == cur.tolist() and int(t_n) == n_free
        assert np.array_equal(t_table.cpu().numpy(), table) and np.array_equal(t_free.cpu().numpy(), free)
        assert slots[k].tolist()[:len(w[4])] == [int(table[b, j // ps]) * ps + j % ps for b, j in w[4]]
    assert step.get_error() == ftd.FTD_OK
    step.close()


def test_refusals():
    import torch
    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    paged, flat = make(3, 256, 128, 8), make(3, 256)
    n = ftd.ftd_kernel_launches()
    ok = dict(old_lens=z(3), new_lens=z(3), served=z(3), block_table=z((3, 2)), free_pages=z(8), n_free=z(1))
    both = z(64)
    bad = [dict(block_table=None), dict(free_pages=None), dict(n_free=None), dict(served=ok["free_pages"][:3]),
           dict(n_free_out=ok["old_lens"][:1]), dict(offsets=ok["old_lens"]), dict(slots=both, positions=both),
           dict(slots=both[:40], positions=both[24:]), dict(offsets=ok["block_table"].view(-1)[:4])]
    for kw in bad:
        with pytest.raises((ftd.FtdError, ValueError)):
            paged.tables(**dict(ok, **kw))
    with pytest.raises(ftd.FtdError):
        flat.tables(**ok)
    L = ftd.load_library()
    p = lambda t: t.data_ptr()  # noqa: E731
    a, b, c = p(ok["old_lens"]), p(ok["new_lens"]), p(ok["served"])
    t, f, m = p(ok["block_table"]), p(ok["free_pages"]), p(ok["n_free"])
    for args in ((0, b, c, t, f, m, 0, 0, 0, 0, 0), (a, 0, c, t, f, m, 0, 0, 0, 0, 0), (a, b, 0, t, f, m, 0, 0, 0, 0, 0),
                 (a + 2, b, c, t, f, m, 0, 0, 0, 0, 0), (a, b, c, t + 1, f, m, 0, 0, 0, 0, 0), (a, b, c, t, f, m, 0, 0, 0, 0, -1),
                 (a, b, c, t, f, m, 0, 0, 0, 0, 1 << 31), (a, b, a + 4, t, f, m, 0, 0, 0, 0, 0)):
        assert L.ftd_build_tables(paged.ctx, *args, 0) == ftd.FTD_ERR_INVALID_ARG, args
    assert ftd.ftd_kernel_launches() == n
    paged.close(), flat.close()
