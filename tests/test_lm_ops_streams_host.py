"""Which stream the Python calls of the operators around the head allocate and launch on, against a library and an
allocator that only take notes (no GPU)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from centroid_masked_sparse_gb300 import lm_ops

GPU = torch.device("cuda", 0)


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    is_cuda, device = True, GPU
    noted = []

    def get_device(self):
        return 0

    def record_stream(self, stream):
        OnGpu.noted.append(("record", self.data_ptr(), stream))


class Stream:
    cuda_stream = 0x5117


@pytest.fixture
def notes(monkeypatch):
    """("alloc" or "launch", stream or None) in order; addresses of tensors recorded on a stream."""
    seen, current = [], [None]

    @contextlib.contextmanager
    def enter(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    def allocate(make):
        def call(*shape, dtype=None, device=None):
            seen.append(("alloc", current[0]))
            return make(*shape, dtype=dtype).as_subclass(OnGpu)
        return call

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_bytes"):
                    return 1024
                seen.append(("launch", Stream if args[-1] == Stream.cuda_stream else None))
                return 0
            return call

    monkeypatch.setattr(lm_ops, "lib", Library)
    monkeypatch.setattr(lm_ops, "_raw_stream", lambda index: current[0].cuda_stream if current[0] else 0)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch, "empty", allocate(torch.empty))
    monkeypatch.setattr(torch, "zeros", allocate(torch.zeros))
    OnGpu.noted.clear()
    return seen


def gpu(*shape, dtype=torch.bfloat16):
    return torch.ones(*shape, dtype=dtype).as_subclass(OnGpu)


def calls():
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32

    def weight():
        return lm_ops.Q4Weight(gpu(16, 32, dtype=u8), gpu(16, 1))

    def cache():
        return lm_ops.KvCache(gpu(4, 1, 16, 64, dtype=u8), gpu(4, 1, 16, 64, dtype=u8), gpu(4, 1, dtype=f32), gpu(4, 1, dtype=f32))

    table, lengths = gpu(2, 2, dtype=i32), gpu(2, dtype=i32)
    logits, tokens, stats = gpu(3, 50, dtype=f32), gpu(3, dtype=i32), gpu(3, dtype=f32)
    return {
        "quantize": (weight, lambda _, **s: lm_ops.Q4Weight.quantize(gpu(16, 64), **s)),
        "mtp_q4_quantize": (weight, lambda _, **s: lm_ops.mtp_q4_quantize(gpu(16, 64), 64, True, **s)),
        "Q4Weight": (weight, lambda _, **s: lm_ops.Q4Weight(gpu(16, 32, dtype=u8), gpu(16, 1), **s)),
        "mtp_q4_matvec": (weight, lambda w, **s: lm_ops.mtp_q4_matvec(w, gpu(2, 64), **s)),
        "mtp_kv_append": (cache, lambda c, **s: lm_ops.mtp_kv_append(c, table, lengths, gpu(2, 1, 64), gpu(2, 1, 64), **s)),
        "mtp_kv_attention": (cache, lambda c, **s: lm_ops.mtp_kv_attention(c, table, lengths, gpu(2, 1, 64), **s)),
        "mtp_token_logprobs": (weight, lambda _, **s: lm_ops.mtp_token_logprobs(logits, tokens, top=2, **s)),
        "mtp_token_logprobs_backward": (weight, lambda _, **s: lm_ops.mtp_token_logprobs_backward(logits, tokens, stats, stats, stats, **s)),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_allocations_belong_to_the_stream_of_the_launch(notes, name):
    make, call = calls()[name]
    with_it = make()
    for stream in (None, Stream):
        notes.clear()
        call(with_it, **({} if stream is None else {"stream": stream}))
        assert ("launch", stream) in notes and {s for _, s in notes} == {stream}, notes


def test_what_a_weight_is_made_from_is_kept_for_its_stream(notes):
    codes, scales, zeros = gpu(16, 32, dtype=torch.uint8), gpu(16, 1), gpu(16, 1, dtype=torch.uint8)
    lm_ops.Q4Weight(codes, scales, zeros)
    assert not OnGpu.noted
    lm_ops.Q4Weight(codes, scales, zeros, stream=Stream)
    assert {n[1:] for n in OnGpu.noted} == {(t.data_ptr(), Stream) for t in (codes, scales, zeros)}


def test_tensors_off_the_gpu_are_refused(notes):
    """Before anything is allocated or launched, also with a stream."""
    bf16, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    codes, scales = torch.ones(16, 32, dtype=u8), torch.ones(16, 1, dtype=bf16)
    for call in (lambda: lm_ops.Q4Weight(codes, scales),
                 lambda: lm_ops.Q4Weight(codes, scales, stream=Stream),
                 lambda: lm_ops.mtp_q4_quantize(torch.ones(16, 64, dtype=bf16)),
                 lambda: lm_ops.Q4Weight.quantize(torch.ones(16, 64, dtype=bf16), stream=Stream),
                 lambda: lm_ops.KvCache(*(torch.ones(4, 1, 16, 64, dtype=u8) for _ in range(2)), *(torch.ones(4, 1, dtype=f32) for _ in range(2)))):
        with pytest.raises(AssertionError, match="on a GPU"):
            call()
    assert not notes


def test_workspaces_of_another_kind_are_refused(notes):
    cache, call = calls()["mtp_kv_attention"]
    cache = cache()
    notes.clear()
    for workspace in (torch.ones(4096, dtype=torch.uint8), gpu(4096, dtype=torch.int32), gpu(64, 64, dtype=torch.uint8).t()):
        with pytest.raises(AssertionError, match="workspace"):
            call(cache, workspace=workspace)
    assert all(kind == "alloc" for kind, _ in notes)
    call(cache, workspace=gpu(4096, dtype=torch.uint8))
    assert notes[-1] == ("launch", None)
