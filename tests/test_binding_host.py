"""The binding's prepared calls on the host: marshalled, never launched."""
import ctypes
import os

import pytest
import torch

from sparse_embedding_lookup_amd import ctr

class Recorded(torch.Tensor):
    def record_stream(self, stream):
        self.streams = getattr(self, "streams", []) + [stream]


class Stream:
    cuda_stream = 0x100


F, I = torch.zeros, torch.int32


def prepared():
    if not os.path.exists(ctr.LIB_PATH):
        from sparse_embedding_lookup_amd import build
        build.build()
    p = dict(prepare=True)
    offsets, one = torch.arange(5, dtype=torch.int64), F(1, dtype=I)
    grad, src = F(4, 16), F(8, 4, dtype=I)
    return [
        ctr.ctr_unique_ids(torch.arange(8), **p),
        ctr.ctr_embbag_fwd(F(9, 16), torch.arange(8), offsets, 4, 1, F(4, 16), 16, 0, **p),
        ctr.ctr_embbag_bwd(grad, 16, 0, offsets, 4, 1, 16, F(8, dtype=I), F(8, dtype=I), one, **p),
        ctr.ctr_embbag_bwd(grad.bfloat16(), 16, 0, offsets, 4, 1, 16, None, None, one,
                           sorted_src=src, **p),
        ctr.ctr_embbag_bwd_sgd(grad, 16, 0, offsets, 4, 1, 8, src, one, F(9, 16), F(8), 0.1, **p),
        ctr.ctr_dense_bwd_sgd(F(8, 16), F(4, 16), F(4), True, F(8, 4), F(8, 4), 0.1, **p)]


@pytest.mark.parametrize("which", range(6))
def test_prepared_call_keeps_the_workspace_it_was_made_with(which):
    """A workspace that the binding allocated lives as long as the call that writes to it."""
    call = prepared()[which]
    addresses = [a.value for a in call.args if isinstance(a, ctypes.c_void_p)]
    kept = [t for t in ctr._tensors(call.keep) if t.dtype == torch.uint8]
    assert len(kept) == 1 and kept[0].data_ptr() in addresses, call.name


def test_immediate_call_on_a_stream_records_what_it_leaves(monkeypatch):
    """Outputs and the workspace of a call on a given stream may be dropped before it has run."""
    class Lib:
        @staticmethod
        def ctr_logistic_ne(*args):
            return ctr.CTR_OK
    monkeypatch.setattr(ctr, "_lib", Lib)
    out, room = (F(4).as_subclass(Recorded) for _ in range(2))
    stream = Stream()
    assert ctr._run("ctr_logistic_ne", (), stream, False, (out, None), room) == (out, None)
    assert out.streams == [stream] and room.streams == [stream]
