"""Ring all-reduce over p virtual ranks held in one GB300's HBM.

A thin Python binding over the C-ABI library ``librar.so`` (include/rar.h);
all work runs in that library's CUDA kernels.  PyTorch is only used to hand
over device pointers and streams.

    import ring_all_reduce_rar_gb300 as rar
    with rar.Handle(device=0, engine="fused") as h:
        h.allreduce(tensors, op="sum")     # tensors: p CUDA tensors of n elements
        x = h.embedding(tables, tokens)    # a table in p pieces
        r = h.add_rmsnorm(parts, weight, residual=x)     # p ranks' partial results
        y = h.vocab_xent(r.out, pieces, targets, grad=True)  # a vocabulary in p pieces
        s = h.vocab_logprobs(r.out, pieces, tokens, top=5)   # what the model answers with
        h.grad_clip(grads, max_norm=1.0)                     # all ranks' gradients
"""
from ._abi import (DTYPE_CODES, ENGINE_CODES, FAULT_CODES, OP_CODES, RAR_MAX_P, STATUS_NAMES, Handle, Options,
                   RarError, library_path, load_library, make_options, rar_all_gather, rar_allreduce,
                   rar_allreduce_host, rar_allreduce_noalloc, rar_allreduce_ptrs, rar_allreduce_range, rar_debug_set_epoch,
                   rar_destroy,
                   rar_init, rar_last_error, rar_reduce_scatter, rar_send_counts, rar_set_options, rar_status,
                   rar_trace, rar_version)
from ._build import build
from ._ops import (AddRmsNorm, GradNorm, VocabLogprobs, VocabXent, rar_add_rmsnorm, rar_add_rmsnorm_grad, rar_embedding,
                   rar_embedding_grad, rar_grad_clip, rar_grad_norm, rar_vocab_logprobs, rar_vocab_logprobs_grad,
                   rar_vocab_xent)

__all__ = [
    "DTYPE_CODES", "ENGINE_CODES", "FAULT_CODES", "OP_CODES", "RAR_MAX_P", "STATUS_NAMES", "Handle", "Options",
    "RarError", "AddRmsNorm", "VocabXent", "build", "library_path", "load_library", "make_options", "rar_all_gather", "rar_allreduce",
    "rar_allreduce_host", "rar_allreduce_noalloc", "rar_allreduce_ptrs", "rar_allreduce_range", "rar_debug_set_epoch",
    "rar_destroy",
    "rar_init", "rar_last_error", "rar_reduce_scatter", "rar_send_counts", "rar_set_options", "rar_status",
    "rar_trace", "rar_version", "rar_add_rmsnorm", "rar_add_rmsnorm_grad", "rar_embedding", "rar_embedding_grad",
    "rar_vocab_xent", "GradNorm", "VocabLogprobs", "rar_grad_clip", "rar_grad_norm", "rar_vocab_logprobs",
    "rar_vocab_logprobs_grad",
]
