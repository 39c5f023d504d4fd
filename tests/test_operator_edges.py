"""Edges of the prompt, shared-prefix and page operators that need no GPU:
scratch sizes, and where the buffers of a call come from."""
import ctypes
import os

import pytest

from tiered_kv_cache_split_gb300 import _lib as L


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from tiered_kv_cache_split_gb300 import build
        build.build()
    return L.load()


def prefix_scratch(lib, dt, hq, hkv, d, counts, shared, alpha):
    n = ctypes.c_size_t()
    c = (ctypes.c_int32 * len(counts))(*counts)
    L.check(lib.tkv_shared_prefix_attention_scratch_size(len(counts), hq, hkv, d, dt, c, max(counts), shared, alpha, ctypes.byref(n)))
    return n.value


@pytest.mark.parametrize("hq,hkv,d", [(28, 4, 128), (8, 2, 64), (32, 32, 128), (64, 1, 64)])
@pytest.mark.parametrize("counts,shared", [([256] * 64, 256), ([16] * 31, 16), ([1], 1), ([300] * 3, 300), ([9, 300, 9], 9)])
def test_alpha_has_room_for_its_sums_of_weights(lib, hq, hkv, d, counts, shared):
    """A bf16 call with alpha keeps one more float per partial row, with or
    without pages behind the prefix (beside the logits of those pages)."""
    without = prefix_scratch(lib, L.DTYPE_BF16, hq, hkv, d, counts, shared, 0)
    rows = (without - 768) // (4 * (d + 2))        # at least: three columns are rounded up to 256 bytes
    own = sum(n - shared for n in counts) * 16 * hq
    with_alpha = prefix_scratch(lib, L.DTYPE_BF16, hq, hkv, d, counts, shared, 1)
    assert with_alpha - without >= 4 * (rows + own)
    assert rows > 0
    # fp32 keeps one sum for both uses
    with_alpha, without = (prefix_scratch(lib, L.DTYPE_F32, hq, hkv, d, counts, shared, a) for a in (1, 0))
    assert 4 * own <= with_alpha - without < 4 * own + 256


def prompt_scratch(lib, dt, q_lens, k_lens, hq, hkv, d):
    n = ctypes.c_size_t()
    a, b = ((ctypes.c_int32 * len(x))(*x) for x in (q_lens, k_lens))
    L.check(lib.tkv_prompt_attention_scratch_size(len(q_lens), a, b, hq, hkv, d, dt, ctypes.byref(n)))
    return n.value


@pytest.mark.parametrize("dt", [L.DTYPE_BF16, L.DTYPE_F32])
def test_key_ranges_of_a_prompt_end_after_two_to_the_eighteen_keys(lib, dt):
    """So many rows that nothing is gained by splitting keys: partials appear only
    where one sum would pass 2^18 of them, of four waves of tiles at a time."""
    rows = 8 * (19456 if dt == L.DTYPE_BF16 else 9728)
    for keys in (1 << 16, 1 << 18, (1 << 18) + 1, 1 << 20, 1 << 26):
        ranges = -(-keys // (1 << 18))
        got = prompt_scratch(lib, dt, [76 * 256], [keys], 8, 8, 64)
        assert got == 0 if ranges == 1 else 0 <= got - ranges * rows * 4 * (64 + 2) <= 1024


def test_long_prompts_take_turns_over_the_partials(lib):
    """Whole documents: the scratch is that of four waves of tiles, not of all rows."""
    for tokens in (1 << 19, 1 << 20, 1 << 22):
        rows = 4 * 152 * 256 + 8 * 256                       # the waves, and what tiles leave empty
        assert 0 < prompt_scratch(lib, L.DTYPE_BF16, [tokens], [tokens], 32, 8, 128) <= tokens // (1 << 18) * rows * 4 * (128 + 2) + 4096
        # two of them take turns of half the length
        both = prompt_scratch(lib, L.DTYPE_BF16, [tokens, tokens], [tokens, tokens], 32, 8, 128)
        assert both <= tokens // (1 << 18) * (rows + 8 * 256) * 4 * (128 + 2) + 4096
    # beside them, short prompts need nothing, and a chunk behind a long cache what it needs alone
    alone = prompt_scratch(lib, L.DTYPE_BF16, [1 << 20], [1 << 20], 32, 8, 128)
    assert prompt_scratch(lib, L.DTYPE_BF16, [9000, 1 << 20, 300], [9000, 1 << 20, 300], 32, 8, 128) == alone


class FakeStreams:
    """torch.cuda as far as buffers for a call on another stream need it."""

    def __init__(self, monkeypatch):
        import contextlib

        from tiered_kv_cache_split_gb300 import operators    # its torch is everyone's
        self.now, self.made, self.recorded = "current", [], []

        @contextlib.contextmanager
        def stream(s):
            before, self.now = self.now, s
            yield
            self.now = before

        class Tensor:
            def record_stream(me, s):
                self.recorded.append(s)

            def data_ptr(me):
                return 0

        def empty(*a, **k):
            self.made.append(self.now)
            return Tensor()

        monkeypatch.setattr(operators.torch.cuda, "stream", stream)
        monkeypatch.setattr(operators.torch.cuda, "current_stream", lambda *a: self.now)
        monkeypatch.setattr(operators.torch, "empty", empty)
        self.on = object.__new__(operators._On)
        self.on.device, self.on.guard, self.on.given, self.on.raw = 0, None, "side", 1


def test_buffers_of_a_call_come_from_its_streams_memory(monkeypatch):
    """A block of the current stream's memory may be one that a tensor just gave
    back while work queued on the current stream still uses it: nothing orders
    another stream behind that work."""
    f = FakeStreams(monkeypatch)
    f.on.empty(4, "dtype")
    f.on.scratch(None, 1024)
    assert f.made == ["side", "side"]
    assert f.recorded == ["current"]        # what is returned outlives its use on the caller's stream
    assert f.now == "current"


def test_buffers_of_the_other_stateless_calls_too(monkeypatch):
    from tiered_kv_cache_split_gb300 import cache
    f = FakeStreams(monkeypatch)
    cache._empty("side", 4, "dtype", "device")
    assert f.made == ["side"] and f.recorded == ["current"]
    cache._empty(None, 4, "dtype", "device")
    assert f.made == ["side", "current"] and f.recorded == ["current"]


def test_tensors_that_ask_for_a_gradient_are_refused():
    """The operators have no backward pass: an output without history would end
    a gradient's way without a word."""
    import torch

    import tiered_kv_cache_split_gb300 as t
    x = [torch.zeros(6, h, 64) for h in (4, 2, 2)]
    for i in range(3):
        y = list(x)
        y[i] = x[i].clone().requires_grad_()
        with pytest.raises(ValueError, match="q, k, v: the operator has no backward pass"):
            t.prompt_attention(*y, [6])
        for again in (y[i] * 2, y[i].detach()):
            y[i] = again
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # as far as a CPU tensor gets
                t.prompt_attention(*y, [6])
    q, pool = torch.zeros(3, 4, 64), torch.zeros(9, 2, 2, 16, 64)
    table, mask = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    for a, b in ((q.clone().requires_grad_(), pool), (q, pool.clone().requires_grad_())):
        with pytest.raises(ValueError, match="q, pool: the operator has no backward pass"):
            t.shared_prefix_attention(a, b, table, mask, [1] * 3, 0)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            t.shared_prefix_attention(a, b, table, mask, [1] * 3, 0)


def test_arguments_of_another_type_are_named():
    import numpy as np
    import torch

    import tiered_kv_cache_split_gb300 as t
    q, pool = torch.zeros(3, 4, 64), torch.zeros(9, 2, 2, 16, 64)
    table, mask, refs = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(9, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    good = dict(q=q, pool=pool, page_table=table, slot_mask=mask, page_counts=[1] * 3, shared_pages=0)
    for name, bad in (("q", None), ("q", q.numpy()), ("pool", None), ("pool", [1]), ("page_table", table.numpy()), ("page_table", None),
                      ("slot_mask", None), ("page_counts", None), ("page_counts", [1.0] * 3), ("page_counts", torch.ones(3)),
                      ("page_counts", [2 ** 31] * 3), ("shared_pages", 1.5), ("shared_pages", None), ("shared_pages", "1")):
        with pytest.raises(ValueError, match=name):
            t.shared_prefix_attention(**{**good, name: bad})
    for counts in (np.array([1, 1, 1]), torch.ones(3, dtype=torch.int64), (1, 1, 1)):      # these are host ints: the device is next
        with pytest.raises(ValueError, match="CUDA"):
            t.shared_prefix_attention(**{**good, "page_counts": counts, "shared_pages": np.int64(0)})
    k = torch.zeros(6, 2, 64)
    for name, bad in (("q", None), ("k", k.numpy()), ("v", None), ("q_lens", None), ("q_lens", 6), ("q_lens", [6.0]), ("k_lens", "6")):
        with pytest.raises(ValueError, match=name):
            t.prompt_attention(**{**dict(q=torch.zeros(6, 4, 64), k=k, v=k, q_lens=[6], k_lens=[6]), name: bad})
    book = dict(page_table=table, page_counts=[1] * 3, page_refs=refs, slot_mask=mask)
    for name, bad in (("page_table", None), ("page_table", table.numpy()), ("page_refs", None), ("slot_mask", mask.numpy()), ("seqs", None),
                      ("seqs", [0.5])):
        with pytest.raises(ValueError, match=name):
            t.free_sequences(**{**book, "seqs": [0], name: bad})
        if name != "seqs":
            for call, more in ((t.fork_sequences, dict(parents=[0], children=[1])), (t.compact_sequences, {})):
                if name != "page_refs":
                    with pytest.raises(ValueError, match=name):
                        call(**{**book, "pool": pool, **more, name: bad})
    for call, more in ((t.fork_sequences, dict(parents=[0], children=[1])), (t.compact_sequences, {})):
        for bad in (None, pool.numpy(), pool[0], pool[..., ::2]):
            with pytest.raises(ValueError, match="pool"):
                call(**{**book, "pool": bad, **more})


def test_a_stream_of_another_type_is_named(monkeypatch):
    from tiered_kv_cache_split_gb300 import operators
    monkeypatch.setattr(operators, "_current_device", lambda: 0)
    monkeypatch.setattr(operators, "_raw_stream", lambda i: 0)
    for bad in (0, "side", object()):
        with pytest.raises(ValueError, match="stream"):
            operators._On(0, bad)
