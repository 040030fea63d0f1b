"""What BlockAttention and Sampler refuse of the arrays that the library takes by their addresses (no GPU: each call is
refused before anything is enqueued)."""
import pytest
import torch

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def T():
    from draft_head_gb300 import build
    build.build()
    from draft_head_gb300 import target
    return target


def layer(T, batch=3, dtype=BF, **kw):
    k = torch.zeros(batch, 2, 20, 64, dtype=dtype)
    return T.BlockAttention(k, torch.zeros_like(k), n_q_heads=4, max_tokens=12, max_q=4, max_ctx=16, **kw)


def ints(*x, dtype=I32):
    return torch.tensor(x, dtype=dtype)


CTX, START, POS = ints(1, 2, 3), ints(0, 4, 8, 12), torch.arange(12, dtype=I32)
BAD_ROWS = [
    dict(ctx_len=ints(1, 2, 3, dtype=torch.int64)), dict(ctx_len=ints(1, 2)), dict(ctx_len=ints(1, 1).repeat(3)[::2]),
    dict(ctx_len=CTX[:1].expand(3)), dict(ctx_len=CTX.float()),
    dict(q_start=ints(0, 4, 8, 12, dtype=torch.int64)), dict(q_start=ints(0, 4, 8)), dict(q_start=START.repeat(2)[::2]),
    dict(positions=POS.long()), dict(positions=POS[:11]), dict(positions=POS.repeat(2)[::2]), dict(positions=POS.short()),
]


@pytest.mark.parametrize("i", range(len(BAD_ROWS)))
def test_lengths_and_positions_that_are_refused(T, i):
    p = layer(T)
    a = dict(ctx_len=CTX, q_start=START, positions=POS)
    a.update(BAD_ROWS[i])
    with pytest.raises(ValueError, match=next(iter(BAD_ROWS[i]))):
        p.append(torch.zeros(12, 8 * 64, dtype=BF), **a)
    with pytest.raises(ValueError, match=next(iter(BAD_ROWS[i]))):
        p.attend(torch.zeros(12, 4, 64, dtype=BF), **a)


@pytest.mark.parametrize("name", ["ctx_len", "q_start", "positions"])
def test_arrays_on_another_device_are_refused(T, name):
    p = layer(T)
    p.ordinal = 0  # a cache on the first GPU

    class OnGpu:  # an array as it would look there
        def __init__(self, t):
            self.t, self.dtype, self.shape, self.device = t, t.dtype, t.shape, "cuda:0"
            self.numel, self.is_contiguous, self.data_ptr = t.numel, t.is_contiguous, t.data_ptr

        def get_device(self):
            return 0

    a = {k: v if k == name else OnGpu(v) for k, v in dict(ctx_len=CTX, q_start=START, positions=POS).items()}
    with pytest.raises(ValueError, match=name):
        p.attend(OnGpu(torch.zeros(12, 4, 64, dtype=BF)), **a)


def seen(*shape):
    return torch.ones(*shape, dtype=torch.uint8)


@pytest.mark.parametrize("mask", [seen(4, 4), seen(1, 4, 4), seen(2, 4, 4), seen(3, 3, 4), seen(3, 4, 3), seen(3, 4, 8)[..., ::2],
                                  seen(4, 4).expand(3, 4, 4), torch.tensor(1, dtype=torch.uint8), seen(3, 4, 4).bool(), seen(3, 4, 4).int()])
def test_tree_masks_that_are_refused(T, mask):
    """Among them a mask of one request for three, which the kernels would read past."""
    with pytest.raises(ValueError, match="mask"):
        layer(T).attend(torch.zeros(12, 4, 64, dtype=BF), CTX, q_start=START, mask=mask)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weights_and_tables_that_are_refused(T, dtype):
    """An fp32 weight beside a bf16 cache would be read as twice as many bf16 numbers, a bf16 table past its end."""
    other = F32 if dtype == BF else BF
    for name in ("q_weight", "k_weight"):
        for bad in (torch.ones(64, dtype=other), torch.ones(63, dtype=dtype), torch.ones(128, dtype=dtype)[::2],
                    torch.ones(1, dtype=dtype).expand(64)):
            with pytest.raises(ValueError, match=name):
                layer(T, dtype=dtype, **{name: bad})
        layer(T, dtype=dtype, **{name: torch.ones(64, dtype=dtype)})
    for bad in (torch.ones(30, 64, dtype=BF), torch.ones(30, 64, dtype=torch.float64), torch.ones(64), torch.ones(2, 30, 64),
                torch.ones(30, 128)[:, ::2]):
        with pytest.raises(ValueError, match="rope"):
            layer(T, dtype=dtype, rope=bad)
    layer(T, dtype=dtype, rope=torch.ones(30, 64))


def test_rows_and_caches_on_another_device_are_refused(T):
    p = layer(T)
    p.ordinal = 0
    with pytest.raises(ValueError, match="qkv"):
        p.append(torch.zeros(12, 8 * 64, dtype=BF), CTX, q_start=START)
    with pytest.raises(ValueError, match="^q:"):
        p.attend(torch.zeros(12, 4, 64, dtype=BF), CTX, q_start=START)
    k = torch.zeros(3, 2, 20, 64, dtype=BF)
    with pytest.raises(ValueError, match="one device"):
        T.B.kv_cache(k, torch.empty_like(k, device="meta"))


BAD_DRAWS = [
    dict(gumbel=torch.zeros(4, 50, dtype=BF)), dict(gumbel=torch.zeros(3, 50)), dict(gumbel=torch.zeros(4, 49)),
    dict(gumbel=torch.zeros(4, 100)[:, ::2]), dict(gumbel=torch.zeros(50, 4).T), dict(gumbel=torch.zeros(4, 50, dtype=torch.float64)),
    dict(gumbel=torch.zeros(200)),
    dict(top_k=torch.zeros(4, dtype=torch.int64)), dict(top_k=torch.zeros(3, dtype=I32)), dict(top_k=torch.zeros(8, dtype=I32)[::2]),
    dict(top_k=torch.zeros(4)), dict(temperature=torch.ones(4, dtype=torch.float64)), dict(temperature=torch.ones(1).expand(4)),
    dict(top_p=torch.ones(3)), dict(top_p=torch.ones(4, dtype=BF)), dict(min_p=torch.ones(4, dtype=I32)), dict(min_p=torch.ones(1)),
    dict(logits=torch.zeros(4, 50, 1)), dict(logits=torch.zeros(4, 51)), dict(logits=torch.zeros(5, 50)), dict(logits=torch.zeros(4, 50, dtype=BF)),
]


@pytest.mark.parametrize("i", range(len(BAD_DRAWS)))
def test_noise_and_settings_that_are_refused(T, i):
    """Among them an int64 top-k, which turned the filter off for every other row, and noise of fewer rows than the logits."""
    a = dict(logits=torch.zeros(4, 50), gumbel=torch.zeros(4, 50), temperature=torch.ones(4), top_k=torch.zeros(4, dtype=I32),
             top_p=torch.ones(4), min_p=torch.zeros(4))
    a.update(BAD_DRAWS[i])
    with pytest.raises(ValueError, match=next(iter(BAD_DRAWS[i]))):
        T.Sampler(4, 50, device="cpu").sample(**a)


@pytest.mark.parametrize("name", ["logits", "gumbel"])
def test_logits_and_noise_on_another_device_are_refused(T, name):
    s = T.Sampler(4, 50, device="cpu")
    a = dict(logits=torch.zeros(4, 50), gumbel=torch.zeros(4, 50))
    a[name] = torch.zeros(4, 50, device="meta")
    s.ordinal = 0 if name == "logits" else -1
    if name == "gumbel":  # both look as if they had no device; the noise alone is moved
        class Away:
            def __init__(self, t):
                self.dtype, self.shape, self.device, self.dim, self.stride = t.dtype, t.shape, "cuda:0", t.dim, t.stride

            def get_device(self):
                return 0
        a[name] = Away(torch.zeros(4, 50))
    with pytest.raises(ValueError, match=name):
        s.sample(**a)


@pytest.mark.parametrize("dtype,rows", [(0, 1), (0, 5000), (1, 1), (1, 5000)])
def test_the_longest_vocabulary_is_the_one_that_is_written_down(T, dtype, rows):
    """The largest that the header names is not refused for its size (the launch may be, without a GPU), one more is."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "domino.h")).read()
    most = int(re.search(r"V is at most ([\d,]+)", text).group(1).replace(",", ""))
    f, unsupported = 0x100000, 2  # an address that nothing reads: without a GPU no kernel runs

    def status(V):
        return T.B.lib.domino_sample(dtype, f, V, rows, V, None, None, None, None, f, V, f, None, f, 256, None)

    assert status(most + 1) == unsupported
    if not torch.cuda.is_available():
        assert status(most) not in (0, unsupported)
