"""POET reparameterized linear layer for MI355X (gfx950): HIP kernels behind a C ABI, with a thin Python binding.

Each weight is W = R W0 P with a fixed random W0 and orthogonal R, P built by the truncated Cayley-Neumann
series from skew-symmetric generators, as block-diagonal (POET-BS) or index-sampled (POET-FS) primitives. The
library provides the forward pass, the backward pass to the skew parameters and merge-then-reinitialize, and what a
training or evaluation step needs around the linears: token log-probabilities, distillation and the seam of two blocks.
"""
from .binding import (POET_BF16, POET_BS, POET_DISTILL_RENORM, POET_DISTILL_TAIL, POET_F32, POET_FS,  # noqa: F401
                      POET_MAX_NORM, POET_MAX_TOP, POET_MAX_VOCAB, POET_OP_BUILD, POET_OP_BWD, POET_OP_FWD,
                      POET_OP_MERGE, POET_SIDE_P, POET_SIDE_R, PoetError, layer, lib, poet_block_norm_bwd,
                      poet_block_norm_fwd, poet_block_norm_workspace_bytes, poet_build_orthogonal,
                      poet_build_workspace_bytes, poet_distill, poet_distill_bwd, poet_distill_workspace_bytes,
                      poet_layer, poet_last_error, poet_linear_bwd, poet_linear_fwd, poet_merge, poet_num_prims,
                      poet_powers_len, poet_prim_len, poet_sample_indices, poet_sample_workspace_bytes, poet_side,
                      poet_status_string, poet_theta_len, poet_token_logprobs, poet_token_logprobs_bwd,
                      poet_token_logprobs_workspace_bytes, poet_version, poet_workspace_bytes, side, side_of)
from .layer import PoetLinear  # noqa: F401
