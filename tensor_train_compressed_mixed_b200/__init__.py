"""B200-native embedding tables, Tensor-Train compressed and dense, and their training steps
(libttemb + a thin ctypes binding)."""
from . import abi, dp
from .abi import TTEmbError
from .dense import DenseEmbedding
from .embedding import TTEmbeddingBag, from_workload
from .optim import AdamW

__all__ = ["abi", "dp", "TTEmbError", "AdamW", "DenseEmbedding", "TTEmbeddingBag", "from_workload"]
