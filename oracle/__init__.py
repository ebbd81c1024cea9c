"""CPU oracle package (test infrastructure only; see csffn_oracle's header)."""
from .csffn_oracle import *  # noqa: F401,F403
from .csffn_oracle import RMS_EPS  # noqa: F401
from .moe_oracle import (block_norm, moe_combine, moe_ffn, moe_ffn_parts, moe_ffn_tol_two_parts,  # noqa: F401
                         moe_logits, moe_route, moe_sort)
