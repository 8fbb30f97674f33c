"""Refusals of the attention entry points with tensors on the device: every
check of shape, type, stride, alignment and range is reached by a call that is
right in all else, says what is wrong, and leaves the outputs alone.
"""
import pytest

from harness import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]

torch = pytest.importorskip("torch")
import paged_expert_cache_gb300 as pec  # noqa: E402

T, HQ, HKV, DIM = 4, 8, 2, 64


def bf16(*shape):
    return torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def strided(heads):
    """[T, heads, DIM] with the heads of a row apart."""
    return bf16(T, heads, 2, DIM)[:, :, 0]


def shifted(*shape):
    """A dense tensor 8 bytes past a 16-byte boundary."""
    n = 1
    for s in shape:
        n *= s
    return bf16(n + 4)[4:].view(shape)


def narrow(heads):
    """Rows 4 elements more than a multiple of 8 apart."""
    return bf16(T, heads * DIM + 4)[:, :heads * DIM].unflatten(1, (heads, DIM))


def refused(call, what, *untouched):
    with pytest.raises(pec.MoeError) as e:
        call()
    assert e.value.status == pec.ERR_INVALID and what in str(e.value), str(e.value)
    for t in untouched:
        assert (t == 7.0).all()


PROMPT = [
    (dict(q=lambda: bf16(T, HQ * DIM)), "q, k, v and out must be torch tensors [T, heads, head_dim]"),
    (dict(q=lambda: bf16(T, HQ, DIM).float()), "q must be bfloat16"),
    (dict(k=lambda: bf16(T, HKV, DIM).half()), "k must be bfloat16"),
    (dict(v=lambda: bf16(T - 1, HKV, DIM)), "v has 3 rows, not 4"),
    (dict(k=lambda: bf16(T, HKV, 32)), "k must be [T, 2, 64], got (4, 2, 32)"),
    (dict(v=lambda: bf16(T, HKV, 32)), "v must be [T, 2, 64], got (4, 2, 32)"),
    (dict(v=lambda: bf16(T, HKV + 1, DIM)), "v must be [T, 2, 64], got (4, 3, 64)"),
    (dict(q=lambda: strided(HQ)), "the heads and dims of a row of q must be contiguous"),
    (dict(k=lambda: strided(HKV)), "the heads and dims of a row of k must be contiguous"),
    (dict(v=lambda: bf16(T, HKV, 2 * DIM)[..., ::2]), "the heads and dims of a row of v must be contiguous"),
    (dict(out=lambda: bf16(T, HQ + 1, DIM)[:, :HQ]), "out must be contiguous"),
    (dict(out=lambda: bf16(T + 1, HQ, DIM)), "out has 5 rows, not 4"),
    (dict(out=lambda: bf16(T, HQ, DIM).float()), "out must be bfloat16"),
    (dict(cu_q=lambda: i32(0, T).long()), "cu_q must be a contiguous int32 tensor of 1 dimension(s)"),
    (dict(cu_q=lambda: i32(0, 0, T, T)[::2]), "cu_q must be a contiguous int32 tensor of 1 dimension(s)"),
    (dict(cu_q=lambda: i32(0, T)[None]), "cu_q must be a contiguous int32 tensor of 1 dimension(s)"),
    (dict(cu_k=lambda: i32(0, 1, T)), "cu_k must have shape (2,), got (3,)"),
    (dict(cu_k=lambda: i32(0, T).cpu()), "cu_k must be on the current CUDA device"),
    (dict(cu_q=lambda: i32(0)), "num_seqs must be >= 1"),
    (dict(q=lambda: shifted(T, HQ, DIM)), "16-byte aligned"),
    (dict(v=lambda: shifted(T, HKV, DIM)), "16-byte aligned"),
    (dict(k=lambda: narrow(HKV)), "strides multiples of 8"),
    (dict(k=lambda: bf16(T, 3, DIM), v=lambda: bf16(T, 3, DIM)), "q_heads a multiple of it"),
    (dict(q=lambda: bf16(T, HQ, 32), k=lambda: bf16(T, HKV, 32), v=lambda: bf16(T, HKV, 32), out=lambda: bf16(T, HQ, 32)),
     "head_dim must be 64 or 128"),
    (dict(scale=lambda: -0.5), "scale must be finite and not negative"),
    (dict(scale=lambda: float("nan")), "scale must be finite and not negative"),
]


@pytest.mark.parametrize("change,what", PROMPT, ids=[w[:40] for _, w in PROMPT])
def test_prompt(change, what):
    a = dict(q=bf16(T, HQ, DIM), k=bf16(T, HKV, DIM), v=bf16(T, HKV, DIM), out=bf16(T, HQ, DIM), cu_q=i32(0, T), cu_k=None,
             scale=None)
    right = {**a, "out": torch.empty_like(a["out"])}
    pec.attention_prompt(**right)
    a.update({n: make() for n, make in change.items()})
    refused(lambda: pec.attention_prompt(**a), what, a["out"])


BATCH = [
    (dict(cu_tokens=lambda: i32(0, 2, 4).long()), "cu_tokens must be a contiguous int32 tensor of 1 dimension(s)"),
    (dict(cu_tokens=lambda: i32(0, 4)), "cu_tokens must have shape (3,), got (2,)"),
    (dict(kv_lens=lambda: i32(2, 2).float()), "kv_lens must be a contiguous int32 tensor of 1 dimension(s)"),
    (dict(kv_lens=lambda: i32(2, 9, 2)[::2]), "kv_lens must be a contiguous int32 tensor of 1 dimension(s)"),
    (dict(kv_lens=lambda: i32()), "at least one sequence"),
    (dict(block_table=lambda: i32([0, 1, 2, 3], [4, 5, 6, 7])[:, ::2]), "block_table must be a contiguous int32 tensor of 2"),
    (dict(block_table=lambda: i32([0, 1])), "block_table must have 2 rows of at least one page"),
    (dict(block_table=lambda: i32([], [])), "block_table must have 2 rows of at least one page"),
    (dict(block_table=lambda: i32(0, 1)), "block_table must be a contiguous int32 tensor of 2"),
    (dict(cu_tokens=lambda: i32(0, 2, 4).cpu()), "cu_tokens must be on the current CUDA device"),
]


@pytest.mark.parametrize("change,what", BATCH, ids=[w[:40] for _, w in BATCH])
def test_batch(change, what):
    a = dict(cu_tokens=i32(0, 2, 4), kv_lens=i32(2, 2), block_table=i32([0, 1], [2, 3]))
    pec.KVBatch(**a)
    a.update({n: make() for n, make in change.items()})
    refused(lambda: pec.KVBatch(**a), what)


@pytest.fixture(scope="module")
def cache():
    return pec.KVCache(pec.make_kv_config(2, 4, HQ, HKV, DIM, page_tokens=16))


def batch():
    return pec.KVBatch(i32(0, 2, 4), i32(2, 2), i32([0, 1], [2, 3]))


APPEND = [
    (dict(k=lambda: bf16(T, HKV + 1, DIM)), "k must be [T, 2, 64], got (4, 3, 64)"),
    (dict(k=lambda: bf16(T, HKV, DIM).half()), "k must be bfloat16"),
    (dict(k=lambda: strided(HKV)), "the heads and dims of a row of k must be contiguous"),
    (dict(k=lambda: narrow(HKV)), "strides multiples of 8"),
    (dict(k=lambda: shifted(T, HKV, DIM)), "16-byte aligned"),
    (dict(k=lambda: [1.0]), "k and v must be torch tensors"),
    (dict(v=lambda: bf16(T + 1, HKV, DIM)), "v has 5 rows, not 4"),
    (dict(v=lambda: bf16(T, HKV, 2 * DIM)), "v must be [T, 2, 64], got (4, 2, 128)"),
    (dict(q=lambda: bf16(T, HKV, DIM)), "q must be [T, 8, 64], got (4, 2, 64)"),
    (dict(q=lambda: bf16(T, HQ, DIM).float()), "q must be bfloat16"),
    (dict(q_out=lambda: None), "q needs q_out"),
    (dict(q_out=lambda: bf16(T, HQ + 1, DIM)[:, :HQ]), "q_out must be contiguous"),
    (dict(q_out=lambda: bf16(T - 1, HQ, DIM)), "q_out has 3 rows, not 4"),
    (dict(k_out=lambda: bf16(T, HKV + 1, DIM)[:, :HKV]), "k_out must be contiguous"),
    (dict(k_out=lambda: bf16(T, HKV, DIM).half()), "k_out must be bfloat16"),
    (dict(k_out=lambda: shifted(T, HKV, DIM)), "outputs must be 16-byte aligned"),
    (dict(rope=lambda: torch.zeros(8, DIM, device="cuda").double()), "rope must be contiguous float32 [positions, 64]"),
    (dict(rope=lambda: torch.zeros(8, DIM // 2, device="cuda")), "rope must be contiguous float32 [positions, 64]"),
    (dict(rope=lambda: torch.zeros(16, DIM, device="cuda")[::2]), "rope must be contiguous float32 [positions, 64]"),
    (dict(rope=lambda: torch.zeros(0, DIM, device="cuda")), "rope must be contiguous float32 [positions, 64]"),
    (dict(rope=lambda: torch.zeros(8 * DIM + 2, device="cuda")[2:].view(8, DIM)), "rope and outputs must be 16-byte aligned"),
    (dict(layer=lambda: 2), "layer out of range"),
    (dict(layer=lambda: -1), "layer out of range"),
    (dict(batch=lambda: (1, 2)), "batch must be a KVBatch"),
]


@pytest.mark.parametrize("change,what", APPEND, ids=[w[:40] for _, w in APPEND])
def test_append(cache, change, what):
    a = dict(layer=1, q=bf16(T, HQ, DIM), k=bf16(T, HKV, DIM), v=bf16(T, HKV, DIM), batch=batch(),
             rope=torch.zeros(8, DIM, device="cuda"), q_out=bf16(T, HQ, DIM), k_out=bf16(T, HKV, DIM))
    cache.append(**{**a, "q_out": torch.empty_like(a["q_out"]), "k_out": torch.empty_like(a["k_out"])})
    a.update({n: make() for n, make in change.items()})
    refused(lambda: cache.append(**a), what, *[a[n] for n in ("q_out", "k_out") if a[n] is not None])
    cache.status()


ATTEND = [
    (dict(q=lambda: bf16(T, HQ + 1, DIM)), "q must be [T, 8, 64], got (4, 9, 64)"),
    (dict(q=lambda: bf16(T, HQ, DIM).half()), "q must be bfloat16"),
    (dict(q=lambda: strided(HQ)), "the heads and dims of a row of q must be contiguous"),
    (dict(q=lambda: narrow(HQ)), "q_stride a multiple of 8"),
    (dict(q=lambda: None), "q and out must be torch tensors"),
    (dict(out=lambda: bf16(T + 1, HQ, DIM)), "out has 5 rows, not 4"),
    (dict(out=lambda: bf16(T, HQ + 1, DIM)[:, :HQ]), "out must be contiguous"),
    (dict(out=lambda: bf16(T, HQ, DIM).float()), "out must be bfloat16"),
    (dict(out=lambda: shifted(T, HQ, DIM)), "16-byte aligned"),
    (dict(scale=lambda: float("inf")), "scale must be finite and not negative"),
    (dict(scale=lambda: -1.0), "scale must be finite and not negative"),
    (dict(layer=lambda: 2), "layer out of range"),
]


@pytest.mark.parametrize("change,what", ATTEND, ids=[w[:40] for _, w in ATTEND])
def test_attend(cache, change, what):
    a = dict(layer=0, q=bf16(T, HQ, DIM), batch=batch(), out=bf16(T, HQ, DIM), scale=None)
    cache.attend(**{**a, "out": torch.empty_like(a["out"])})
    a.update({n: make() for n, make in change.items()})
    refused(lambda: cache.attend(**a), what, a["out"])
    cache.status()


READ = [
    (dict(k_out=lambda: bf16(T, HKV + 1, DIM)), "k_out must be [T, 2, 64], got (4, 3, 64)"),
    (dict(k_out=lambda: bf16(T, HKV, DIM).float()), "k_out must be bfloat16"),
    (dict(v_out=lambda: bf16(T - 1, HKV, DIM)), "v_out has 3 rows, not 4"),
    (dict(v_out=lambda: bf16(T, HKV + 1, DIM)[:, :HKV]), "v_out must be contiguous"),
    (dict(v_out=lambda: shifted(T, HKV, DIM)), "16-byte aligned"),
    (dict(v_out=lambda: None), "k_out and v_out must be torch tensors"),
    (dict(layer=lambda: 7), "layer out of range"),
]


@pytest.mark.parametrize("change,what", READ, ids=[w[:40] for _, w in READ])
def test_read(cache, change, what):
    a = dict(layer=0, batch=batch(), k_out=bf16(T, HKV, DIM), v_out=bf16(T, HKV, DIM))
    cache.read(**{**a, "k_out": torch.empty_like(a["k_out"]), "v_out": torch.empty_like(a["v_out"])})
    a.update({n: make() for n, make in change.items()})
    refused(lambda: cache.read(**a), what, *[a[n] for n in ("k_out", "v_out") if a[n] is not None])
    cache.status()


def test_a_closed_cache_is_refused(cache):
    c = pec.KVCache(pec.make_kv_config(1, 4, HQ, HKV, DIM, page_tokens=16))
    c.close()
    out = bf16(T, HQ, DIM)
    refused(lambda: c.attend(0, bf16(T, HQ, DIM), batch(), out), "handle is NULL", out)
