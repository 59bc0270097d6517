"""Layout-aware FSDP2 collective local stages on MI355X (gfx950).

  Plan                   host shard-layout plan (dimension-0 shards, padding)
  reduce_scatter_local   W ranks' bf16 (or fp32) gradients -> W packed fp32
                         shards (with Equation 5's alpha and accumulate)
  reduce_scatter_local_noalloc
                         the same from bf16 gradients, allocating nothing
                         (tables in a fixed device scratch array)
  allgather_copyout      rank-major bf16 buffer -> per-parameter tensors
  allgather_copyin       every rank's fp32/bf16 shards -> rank-major bf16 buffer
  checkpoint_pack, checkpoint_unpack
                         activations kept in 8 bits between the passes
  checkpoint_weight_grad a linear layer's weight gradient from such a
                         checkpoint of its input
  vocab_loss, vocab_loss_grad
                         cross entropy of the output projection without its
                         logits; with its gradients
  stock_chunk_cat        stock FSDP2's gradient pack of one rank (the baseline)
  probe, victim_axpb, Stream
                         interference instruments: hardware-ID probe,
                         elementwise victim, CU-masked streams

The *_call variants check and marshal the tensors once and return a callable
that launches with one library call (for buffers reused every step); where an
operation needs a workspace, each launch takes its own unless it is given one.

The work runs in the HIP library libtide.so (include/tide.h); importing this
package fails if that library has not been built.
"""
from .tide import (  # noqa: F401
    FLAG_CACHED_LOADS,
    FLAG_CACHED_STORES,
    FLAG_NO_LDS,
    MAX_WORLD,
    Plan,
    DTYPE_BF16,
    DTYPE_F32,
    TideError,
    allgather_copyin,
    allgather_copyin_call,
    allgather_copyout,
    allgather_copyout_call,
    checkpoint_layout,
    checkpoint_pack,
    checkpoint_pack_call,
    checkpoint_unpack,
    checkpoint_unpack_call,
    checkpoint_weight_grad,
    checkpoint_weight_grad_call,
    checkpoint_weight_grad_workspace,
    reduce_scatter_call,
    reduce_scatter_local,
    reduce_scatter_local_noalloc,
    stock_chunk_cat,
    stock_chunk_cat_call,
    Stream,
    decode_probe,
    device_info,
    probe,
    victim_axpb,
    vocab_loss,
    vocab_loss_call,
    vocab_loss_grad,
    vocab_loss_grad_call,
    vocab_loss_workspace,
)
