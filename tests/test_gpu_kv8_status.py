"""What a refused call leaves: the cache as it was, and a status that stays until it
is read."""
import pytest
import torch

from tests.test_gpu_kv8 import cu_of, fill, gen, ints, make_cache

pytestmark = pytest.mark.gpu


def bytes_of(c):
    return [t.clone() for t in (c.table, c.lens, c.refs, c.k, c.v, c.kscale, c.vscale)]


def same(c, state):
    return all(torch.equal(a, b) for a, b in zip(state, (c.table, c.lens, c.refs, c.k, c.v, c.kscale, c.vscale)))


def full_pool(tq_lib, dev, fmt="i8"):
    """Two sequences that share both pages of the pool: the second one's next token
    needs a copy that there is no room for."""
    c = make_cache(tq_lib, dev, fmt, layers=2, page=16, slots=3, max_pages=4, pages=2)
    c.reserve(ints([0], dev), ints([20], dev))
    x = torch.randn(20, 2, 128, generator=gen(1)).to(torch.bfloat16).to(dev)
    for layer in range(2):
        c.append(layer, x, x, cu_of([20], dev), 20, slots=ints([0], dev))
    c.fork(ints([0], dev), ints([1], dev))
    c.status()
    return c


def refused(tq_lib, c, what):
    with pytest.raises(tq_lib.TQError) as e:
        c.status()
    assert e.value.status == getattr(tq_lib.binding, "TQ_ERR_" + what)


@pytest.mark.parametrize("new", [1, 12])
def test_a_refused_reserve_stops_the_step(tq_lib, cuda, new):
    """reserve, then append and attention for every layer, then status(): the tokens
    that are there keep their bytes, in pages that others share too."""
    c = full_pool(tq_lib, cuda)
    state = bytes_of(c)
    slots, cu = ints([1], cuda), cu_of([new], cuda)
    x = torch.randn(new, 2, 128, device=cuda).to(torch.bfloat16)
    q = torch.randn(new, 16, 128, device=cuda).to(torch.bfloat16)
    lse = torch.zeros(new, 16, device=cuda)
    for _ in range(2):  # a second step before anybody looks
        c.reserve(slots, ints([new], cuda))
        for layer in range(2):
            c.append(layer, x, x, cu, new, slots=slots)
            out = c.attention(layer, q, cu, new, slots=slots, lse=lse)
    k, v = c.read(0, ints([0], cuda), cu_of([20], cuda), 20, 20)
    c.truncate(ints([0], cuda), ints([3], cuda))
    c.fork(ints([0], cuda), ints([2], cuda))
    c.compact()
    refused(tq_lib, c, "PAGES")
    assert same(c, state)
    assert (out == 0).all() and (lse == -torch.inf).all() and (k == 0).all() and (v == 0).all()
    c.status()  # read once, it is gone, and the cache works again
    c.truncate(ints([0], cuda), ints([0], cuda))
    c.reserve(slots, ints([new], cuda))
    c.append(0, x, x, cu, new, slots=slots)
    out = c.attention(0, q, cu, new, slots=slots)
    c.status()
    assert int(c.lens[1]) == 20 + new and (out != 0).any()


def test_a_refused_reserve_in_a_graph(tq_lib, cuda):
    c = full_pool(tq_lib, cuda)
    slots, one, cu = ints([1], cuda), ints([1], cuda), cu_of([1], cuda)
    x = torch.randn(1, 2, 128, device=cuda).to(torch.bfloat16)
    q = torch.randn(1, 4, 128, device=cuda).to(torch.bfloat16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.reserve(slots, one)
        c.append(0, x, x, cu, 1, slots=slots)
        out = c.attention(0, q, cu, 1, slots=slots)
    state = bytes_of(c)
    for _ in range(3):
        g.replay()
        refused(tq_lib, c, "PAGES")
        assert same(c, state) and (out == 0).all()
    c.truncate(ints([0], cuda), ints([0], cuda))
    g.replay()
    c.status()
    assert int(c.lens[1]) == 21 and (out != 0).any()


def test_the_first_refusal_stands(tq_lib, cuda):
    c = make_cache(tq_lib, cuda, page=16, slots=4, max_pages=4, pages=6)
    c.reserve(ints([0, 1], cuda), ints([20, 16], cuda))
    c.truncate(ints([0, 0], cuda), ints([1, 1], cuda))   # ARG
    c.reserve(ints([2, 3], cuda), ints([64, 64], cuda))  # would be PAGES
    c.reserve(ints([2], cuda), ints([1], cuda))          # would be fine
    refused(tq_lib, c, "ARG")
    assert c.lens.tolist() == [20, 16, 0, 0]
    c.status()


def test_two_caches_keep_statuses_of_their_own(tq_lib, cuda):
    a, b = (make_cache(tq_lib, cuda, page=16, slots=2, max_pages=4, pages=2) for _ in "ab")
    a.reserve(ints([0], cuda), ints([40], cuda))
    b.reserve(ints([0], cuda), ints([30], cuda))
    b.status()
    refused(tq_lib, a, "PAGES")


def test_calls_without_work_leave_no_status(tq_lib, cuda):
    """Empty lists and empty batches do nothing and report nothing."""
    for call in (lambda c: c.reserve(ints([], cuda), ints([], cuda)),
                 lambda c: c.attention(0, torch.zeros(0, 4, 128, dtype=torch.bfloat16, device=cuda),
                                       cu_of([0, 0], cuda), 0)):
        # (memory that the call may be handed holds anything)
        for size in (256, 4096, 1 << 20, 1 << 22, 1 << 24):
            torch.full((size // 4,), -8, dtype=torch.int32, device=cuda)
        c = make_cache(tq_lib, cuda, page=16, slots=2, max_pages=4, pages=2)
        call(c)
        c.status()


def test_a_cache_made_in_inference_mode(tq_lib, cuda):
    with torch.inference_mode():
        c = make_cache(tq_lib, cuda, page=16, slots=2, max_pages=4, pages=2)
    c.reserve(ints([0], cuda), ints([40], cuda))
    refused(tq_lib, c, "PAGES")
    c.status()


def test_status_after_another_stream(tq_lib, cuda):
    """status() sees what a call on any stream found, also one that has not begun."""
    c = make_cache(tq_lib, cuda, page=16, slots=2, max_pages=4, pages=2)
    slots, many, one = ints([0], cuda), ints([40], cuda), ints([1], cuda)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.reserve(slots, one)
    c.status()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
        c.reserve(slots, many)
    refused(tq_lib, c, "PAGES")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        torch.cuda._sleep(200_000_000)
        c.reserve(slots, many)
    with torch.cuda.stream(side):
        g.replay()
    refused(tq_lib, c, "PAGES")


def test_status_while_capturing(tq_lib, cuda):
    """A capture cannot wait: status() says so and leaves the capture as it was."""
    c = make_cache(tq_lib, cuda, page=16, slots=2, max_pages=4, pages=2)
    slots, one = ints([0], cuda), ints([1], cuda)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.reserve(slots, one)
        with pytest.raises(RuntimeError):
            c.status()
    g.replay()
    c.status()
    assert int(c.lens[0]) == 1


def test_the_library_without_a_status_word(tq_lib, cuda):
    """d_status NULL: a page operation's own word tells, and nothing is held back."""
    B = tq_lib.binding
    c = make_cache(tq_lib, cuda, page=16, slots=2, max_pages=4, pages=2)
    c.c.d_status = None
    ws = torch.zeros(B.tq_kv8_workspace_bytes(B.TQ_KV8_OP_PAGES, c.c, 1, 0, 0, 0), dtype=torch.uint8, device=cuda)
    stream = torch.cuda.current_stream().cuda_stream
    slots, many, some = ints([0], cuda), ints([40], cuda), ints([20], cuda)
    for counts, want in ((many, B.TQ_ERR_PAGES), (some, B.TQ_OK)):
        B.tq_kv8_reserve(c.c, 1, slots.data_ptr(), counts.data_ptr(), ws.data_ptr(), ws.numel(), stream)
        assert B.lib.tq_device_status(ws.data_ptr(), stream) == want
    assert c.lens.tolist() == [20, 0]
    c.status()
    x = torch.randn(20, 2, 128, device=cuda)
    B.tq_kv8_append(c.c, 0, 1, slots.data_ptr(), cu_of([20], cuda).data_ptr(), 20, 20, x.data_ptr(),
                    x.data_ptr(), B.TQ_F32, 256, 128, None, stream)
    k, _ = c.read(0, ints([0], cuda), cu_of([20], cuda), 20, 20, dtype=torch.float32)
    assert ((k - x).abs() <= x.abs().max() / 254 * 1.01).all()


def test_a_cache_made_behind_other_work(tq_lib, cuda):
    """A cache over an engine's tensors can be used on any stream at once: its status
    word does not wait for the stream on which it was made."""
    parts = make_cache(tq_lib, cuda, page=16, slots=2, max_pages=4, pages=2)
    slots, one = ints([0], cuda), ints([1], cuda)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # what the word's memory may hold
        torch.full((512,), 0xF8, dtype=torch.uint8, device=cuda)
        torch.full((4,), -1, dtype=torch.int32, device=cuda)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        c = tq_lib.KV8Cache(parts.k, parts.v, parts.kscale, parts.vscale, parts.table, parts.lens, parts.refs)
    c.reserve(slots, one)
    c.status()
    assert int(c.lens[0]) == 1


def test_many_caches(tq_lib, cuda):
    """Each with a status of its own, however many there are, also one made in a
    capture."""
    caches = [make_cache(tq_lib, cuda, page=16, slots=1, max_pages=1, pages=1, d=64) for _ in range(300)]
    assert len({c._status.data_ptr() for c in caches}) == 300
    caches[7].reserve(ints([0], cuda), ints([17], cuda))
    for i, c in enumerate(caches):
        if i == 7:
            refused(tq_lib, c, "ARG")
        else:
            c.status()
    parts, slots, one = caches[0], ints([0], cuda), ints([1], cuda)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = tq_lib.KV8Cache(parts.k, parts.v, parts.kscale, parts.vscale, parts.table, parts.lens, parts.refs)
        c.reserve(slots, one)
    g.replay()
    c.status()
    assert parts.lens.tolist() == [1]
