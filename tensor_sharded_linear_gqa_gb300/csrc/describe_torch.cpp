// describe.c's answers for plain torch tensors, read from the tensor itself: its attributes by way of
// the interpreter cost 0.33 us a tensor (one GB300's host), and a one-token call over eight ranks has
// over thirty tensors. Where torch's headers are missing, describe.c does without.
#include <torch/csrc/autograd/python_variable.h>

#include "tpgqa.h"

namespace {

// tp_dtype, 4 for int32, -1 for any other.
int type_of(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kFloat: return TP_F32;
    case at::kBFloat16: return TP_BF16;
    case at::kFloat8_e4m3fn: return TP_E4M3;
    case at::kByte: return TP_U8;
    case at::kInt: return 4;
    default: return -1;
  }
}

}  // namespace

// 1: described; 0: left to the caller; -1: no plain tensor (a subclass, a stand-in). device: the GPU on which it
// must lie, -1: any; one comparison here, where the attribute costs the interpreter 0.4 us a tensor.
extern "C" int tp_describe_torch(PyObject *o, long dims, int device, tp_tensor *d) {
  if (!THPVariable_CheckExact(o)) return -1;
  try {
    const at::Tensor &t = THPVariable_Unpack(o);
    const int type = type_of(t);
    if (!t.is_cuda() || type < 0 || type > TP_U8 || t.dim() != dims || (device >= 0 && t.get_device() != device)) return 0;
    const auto size = t.sizes(), stride = t.strides();
    const int64_t rows = dims == 2 ? size[0] : 1, cols = size[dims - 1], ld = dims == 2 ? stride[0] : 1;
    if (rows == 0 || cols == 0 || stride[dims - 1] != 1) return 0;
    void *ptr = t.mutable_data_ptr();
    if (ptr == nullptr) return 0;
    // the pitch of a single row is free
    *d = tp_tensor{ptr, type, 0, rows, cols, rows > 1 || ld > cols ? ld : cols};
    return 1;
  } catch (...) {
    return 0;
  }
}

// The address of a contiguous CUDA vector (any shape) of type `type` (as type_of) with n entries (-1: any number),
// 0 where the caller has to look for itself. *bytes receives its size.
extern "C" unsigned long long tp_address_torch(PyObject *o, int type, long long n, int device, unsigned long long *bytes) {
  if (!THPVariable_CheckExact(o)) return 0;
  try {
    const at::Tensor &t = THPVariable_Unpack(o);
    const int64_t have = t.numel();
    if (!t.is_cuda() || (device >= 0 && t.get_device() != device) || (type >= 0 && type_of(t) != type) || have == 0 || (n >= 0 && have != n) || !t.is_contiguous()) return 0;
    *bytes = static_cast<unsigned long long>(have) * t.element_size();
    return reinterpret_cast<unsigned long long>(t.mutable_data_ptr());
  } catch (...) {
    return 0;
  }
}
