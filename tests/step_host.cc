// The Python module of the drafting step's operators on a machine without a
// GPU: linked with its object file in place of libdvl.so and of the few
// PyTorch functions that need a device.  The library's entry points write down
// what they are given; tensors are addresses that nothing reads.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/from_blob.h>
#include <ATen/ops/record_stream_ops.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

#include "dvl.h"

namespace {

int g_device = 0;                    // the current device
c10::StreamId g_stream = 0;          // its current stream's id; the handle is the same number
std::vector<std::string> g_events;   // what was asked for, in order

void event(const std::string &what, uintptr_t stream)
{
    g_events.push_back(what + " device " + std::to_string(g_device) + " stream " +
                       std::to_string(stream));
}

c10::cuda::CUDAStream stream_with(c10::StreamId id, c10::DeviceIndex dev)
{
    return c10::cuda::CUDAStream(c10::cuda::CUDAStream::UNCHECKED,
                                 c10::Stream(c10::Stream::UNSAFE,
                                             c10::Device(c10::DeviceType::CUDA, dev), id));
}

at::Tensor fake(int64_t address, at::IntArrayRef shape, at::ScalarType type, int device)
{
    const c10::Device dev(c10::DeviceType::CUDA, (c10::DeviceIndex)device);
    return at::for_blob(reinterpret_cast<void *>(address), shape)
        .options(at::TensorOptions().dtype(type).device(dev))
        .target_device(dev)
        .make_tensor();
}

}  // namespace

namespace c10::cuda {
DeviceIndex device_count() noexcept { return 4; }
cudaError_t SetDevice(DeviceIndex device, const bool)
{
    g_device = device;
    return cudaSuccess;
}
DeviceIndex ExchangeDevice(DeviceIndex device)
{
    const int was = g_device;
    g_device = device;
    return (DeviceIndex)was;
}
CUDAStream getCurrentCUDAStream(DeviceIndex device) { return stream_with(g_stream, device); }
void setCurrentCUDAStream(CUDAStream s) { g_stream = s.unwrap().id(); }
CUDAStream getStreamFromExternal(cudaStream_t s, DeviceIndex device)
{
    return stream_with(reinterpret_cast<c10::StreamId>(s), device);
}
cudaStream_t CUDAStream::stream() const { return reinterpret_cast<cudaStream_t>(stream_.id()); }
}  // namespace c10::cuda

namespace at::_ops {
Tensor empty_memory_format::call(c10::SymIntArrayRef size, ::std::optional<at::ScalarType> dtype,
                                 ::std::optional<at::Layout>, ::std::optional<at::Device> device,
                                 ::std::optional<bool>, ::std::optional<at::MemoryFormat>)
{
    event("empty", (uintptr_t)g_stream);
    return fake(0x700000, C10_AS_INTARRAYREF_SLOW(size), *dtype, device->index());
}
void record_stream::call(at::Tensor &, at::Stream s) { event("record", (uintptr_t)s.id()); }
}  // namespace at::_ops

extern "C" {
dvl_status dvl_add_rmsnorm(const dvl_norm *, void *s)
{
    event("add_rmsnorm", (uintptr_t)s);
    return DVL_OK;
}
dvl_status dvl_paged_attention(const dvl_kv_cache *, const void *, int64_t, int64_t, int64_t, int32_t,
                               int32_t, int32_t, const int32_t *, int64_t, int32_t, const int32_t *,
                               float, void *, float *, void *, size_t, void *s)
{
    event("paged_attention", (uintptr_t)s);
    return DVL_OK;
}
dvl_status dvl_beam_select(const void *, int32_t, int64_t, int64_t, const float *, int32_t, int32_t,
                           int32_t, int32_t, const int32_t *, float *, int32_t *, int32_t *, void *,
                           size_t, void *s)
{
    event("beam_select", (uintptr_t)s);
    return DVL_OK;
}
dvl_status dvl_beam_reorder(const dvl_state *, int32_t, const dvl_beam_pages *, const dvl_kv_cache *,
                            const int32_t *, int32_t, int32_t, int32_t, void *s)
{
    event("beam_reorder", (uintptr_t)s);
    return DVL_OK;
}
}

namespace {

// tensor(address, shape, dtype, device)
PyObject *py_tensor(PyObject *, PyObject *args)
{
    long long address;
    PyObject *shape, *dtype;
    int device;
    if (!PyArg_ParseTuple(args, "LOOi", &address, &shape, &dtype, &device))
        return nullptr;
    std::vector<int64_t> sizes;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(shape); ++i)
        sizes.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)));
    return THPVariable_Wrap(fake(address, sizes, reinterpret_cast<THPDtype *>(dtype)->scalar_type, device));
}
// state(device, stream): set both, forget the events
PyObject *py_state(PyObject *, PyObject *args)
{
    long long stream;
    if (!PyArg_ParseTuple(args, "iL", &g_device, &stream))
        return nullptr;
    g_stream = stream;
    g_events.clear();
    Py_RETURN_NONE;
}
// events() -> (list, current device, current stream)
PyObject *py_events(PyObject *, PyObject *)
{
    PyObject *list = PyList_New(0);
    for (const std::string &e : g_events) {
        PyObject *s = PyUnicode_FromString(e.c_str());
        PyList_Append(list, s);
        Py_DECREF(s);
    }
    return Py_BuildValue("(NiL)", list, g_device, (long long)g_stream);
}

PyMethodDef methods[] = {{"tensor", py_tensor, METH_VARARGS, nullptr},
                         {"state", py_state, METH_VARARGS, nullptr},
                         {"events", py_events, METH_NOARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "step_host", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_step_host(void) { return PyModule_Create(&module); }
