"""``stream=`` of the Python calls, with work under way on both streams: outputs and
inputs keep their memory until both are done with it, in whatever order the
tensors are freed.  The queues are held up with a spinning kernel, so that what
could meet would meet."""
import pytest
import torch

from copy_write_forked_gb300.dendrite import DendriteError, Pool, Rope

pytestmark = pytest.mark.gpu
N, T, KV, G, D = 2, 64, 2, 4, 128
SPIN = 100_000_000   # some 50 ms


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


@pytest.fixture
def case():
    """A pool with T rows on each of N branches, and what each call on a stream returns with nothing else going on."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    pool = Pool(64, 16, KV, D, torch.bfloat16, max_branches=8)
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = lambda h: torch.randn(N, T, h, D, generator=g, device="cuda").bfloat16()  # noqa: E731
    K, V, Q = rows(KV), rows(KV), rows(KV * G)
    br = [pool.new_branch() for _ in range(N)]
    pool.append_kv(br, K, V)
    rope, parents = Rope(D), list(range(-1, T - 1))

    def rotated(stream=None):
        out = pool.append_rope(br, K, V, rope, Q=Q, stream=stream)
        pool.truncate(br, [T] * N, stream=stream)
        return out

    def split(stream=None):
        pool.append_begin(br, T, stream=stream)
        out = pool.append_layer_rope(0, K, V, rope, Q=Q, stream=stream)
        pool.truncate(br, [T] * N, stream=stream)
        return out

    calls = dict(read=lambda stream=None: pool.read_kv(br, [0] * N, [T] * N, stream=stream)[0], rotated=rotated, split=split,
                 decode=lambda stream=None: pool.tree_attn_decode(Q, br, stream=stream),
                 draft=lambda stream=None: pool.tree_attn_draft(Q, br, parents, stream=stream))
    yield pool, br, calls, (K, V, Q)
    torch.cuda.synchronize()
    pool.close()


NAMES = ["read", "rotated", "split", "decode", "draft"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_freed_on_the_current_stream_with_reads_queued(case, name):
    call = case[2][name]
    want = call()
    torch.cuda.synchronize()
    size = want.numel()
    kept = torch.arange(size, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    copy = torch.zeros_like(kept)
    free = [kept.clone() for _ in range(3)]   # blocks of the outputs' size: whichever is handed out next
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    copies = [copy.clone() for _ in free]
    for c, f in zip(copies, free):
        c.copy_(f)                            # queued behind the spin
    del free, f
    out = call(stream=s)                      # runs at once
    s.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert all(torch.equal(c, kept) for c in copies)


@pytest.mark.parametrize("name", NAMES)
def test_output_freed_while_its_stream_still_writes(case, name):
    call = case[2][name]
    size = call().numel()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    out = call(stream=s)                      # queued behind the spin
    del out
    new = [torch.full((size,), 3.0, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    torch.cuda.synchronize()
    assert all((x == 3.0).all() for x in new)


@pytest.mark.parametrize("name", NAMES)
def test_output_read_on_the_current_stream_and_freed(case, name):
    call = case[2][name]
    want = call().clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(SPIN)
    copy = torch.empty_like(want)
    copy.copy_(out)                           # queued behind the spin
    del out
    with torch.cuda.stream(s):
        new = [torch.full((want.numel(),), 3.0, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(new) == 4


@pytest.mark.parametrize("name", ["append", "layer", "rotated", "decode"])
def test_inputs_freed_while_the_stream_still_reads(case, name):
    pool, br, _, (K, V, Q) = case
    want = pool.tree_attn_decode(Q, br)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    k, v, q = K.clone(), V.clone(), Q.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    if name == "append":
        pool.append_kv(br, k, v, stream=s)
    elif name == "layer":
        pool.append_begin(br, T, stream=s)
        pool.append_layer(0, k, v, stream=s)
    elif name == "rotated":
        pool.append_rope(br, k, v, Rope(D, inv_freq=[0.0] * 64), Q=q, stream=s)
    else:
        out = pool.tree_attn_decode(q, br, stream=s)
    del k, v, q
    new = [torch.full_like(x, 3.0) for x in (K, V, Q) for _ in range(3)]
    torch.cuda.synchronize()
    if name == "decode":
        assert torch.equal(out, want)
    else:
        got = pool.read_kv(br, [T] * N, [T] * N)
        assert torch.equal(got[0].view_as(K), K) and torch.equal(got[1].view_as(V), V)
    assert len(new) == 9


def test_read_kv_into_given_tensors(case):
    pool, br, _, (K, V, _) = case
    k, v = torch.zeros_like(K).view(N * T, KV, D), torch.zeros_like(V).view(N * T, KV, D)
    a, b = pool.read_kv(br, [0] * N, [T] * N, out=(k, v))
    assert a is k and b is v
    pool.sync()
    assert torch.equal(k.view_as(K), K) and torch.equal(v.view_as(V), V)
    for bad in ((k[1:], v[1:]), (k, v.float()), (k, v.cpu()), (k, k), (k.transpose(0, 1), v)):
        with pytest.raises(DendriteError):
            pool.read_kv(br, [0] * N, [T] * N, out=bad)
